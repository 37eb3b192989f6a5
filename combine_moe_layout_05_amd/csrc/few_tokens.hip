// The whole expert layer for a few tokens in two kernels on gfx950, from the
// tokens' rows and their routing to the combined output, with no layout, no
// permuted rows and no copy back to token order:
//   h[p] = act(x[t] Wg^T) * (x[t] Wu^T)        p = t K + k, with the weights of
//   y[t] = sum over k of s[p] * (h[p] Wd^T)    expert ids[p]
//
// Every workgroup reads the ids (at most 512) and finds the experts in use by
// itself. The first kernel takes 64 rows of one expert's [Wg; Wu] and 16 or 32 of
// its slots at a time, the sum split over the wavefronts; the second 16 columns
// of y, its wavefronts one expert (or a part of its sum) after the other, so that
// the slots' results meet in its LDS and are summed there in slot order, fp32:
// no atomics, equal calls give equal bits.
//
// h goes between the kernels as two bf16, the rounded number and what the
// rounding left, 16 bits of significand: the matrix cores take both as rows of
// one product, whose 16 places a few tokens leave empty anyway, so the second
// rounding that a bf16 h would bring costs nothing to avoid. Its rows lie in the
// order of their experts, and in steps of the second kernel's sum: for each step
// and row 32 rounded elements, their 32 rests, the next 32 and so on, so that the
// loads of few or many rows all take whole cache lines.
//
// Bound: the bytes of the weights in use, read once per 16 (first kernel) or 8
// slots of an expert, straight into the registers the matrix cores read; with 4 bits
// also the load instructions, of which a CU takes one in some 30 cycles. Measured on
// MI355X, 256 experts of 7168 -> 2048, 8 per token, us for both kernels: one token 127
// (705 MB, 5.5 TB/s), in 4 bits 40 (187 MB, 4.7 TB/s), of which the start and end of
// the two launches are some 12; 16 tokens 1512 and 375. Where an expert has several
// slots the separate calls read its weights fewer times: with these experts they are
// level at 4 tokens in bf16 (455 us) and ahead from 16 on (1457), in 4 bits ahead at 64
// (796 against 818) and not at 32 (598 against 587); 64 tokens x 2 on 8 experts of 4096
// -> 4096 take 227 us here and 163 there, in 4 bits 109 and 70.
#include "expert_kernels.h"
#include "expert_mma.h"
#include "expert_mxfp4.h"
#include "layer_kernels.h"

#include <type_traits>

namespace moe {
namespace {

constexpr int kMaxWords = 32;           // of a bit per expert (1024)

// What a step of the sum takes from memory for one 16-feature block; the scales
// of 4-bit weights come apart from them.
template <bool FOUR>
struct Weights;
template <>
struct Weights<true> {
    v4i q;
    __device__ bf16x8 frag(int s, uint32_t scale) const { return Mxfp4Step{q, scale}.frag(s); }
};
template <>
struct Weights<false> {
    v4i q[2];
    __device__ bf16x8 frag(int s, uint32_t) const { return __builtin_bit_cast(bf16x8, q[s]); }
};
template <bool FOUR>
struct Step {
    static constexpr int kElems = FOUR ? kMxfp4Step : 64;
    static constexpr int kProducts = kElems / 32;
};

// A block of 16 features: uniform addresses, and the lane's offsets from them.
template <bool FOUR>
struct Block {
    const char* q;
    // Lane (i, g)'s offsets, the same for all blocks of a kernel but for a
    // clamped row.
    static __device__ uint32_t offset(int lane, int32_t row, int64_t pitch) {
        return FOUR ? lane * 16 : static_cast<uint32_t>(row * pitch) + (lane >> 4) * 16;
    }
    __device__ __forceinline__ void load(int32_t t, uint32_t at, int lane, Weights<FOUR>& d) const {
        reform(at);
        if constexpr (FOUR) {
            d.q = __builtin_nontemporal_load(
                reinterpret_cast<const v4i*>(q + int64_t(t) * 1024 + at));
        } else {
#pragma unroll
            for (int s = 0; s < 2; ++s)
                d.q[s] = *reinterpret_cast<const v4i*>(q + (int64_t(t) * 128 + s * 64) + at);
        }
    }
    // The last step of a sum that ends inside it; `left` 8-element chunks are
    // there. Packed weights hold zeros behind them.
    __device__ __forceinline__ void load_last(int32_t t, int left, uint32_t at, int lane,
                                              Weights<FOUR>& d) const {
        if constexpr (FOUR) {
            load(t, at, lane, d);
        } else {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                d.q[s] = v4i{0, 0, 0, 0};
                if (4 * s + (lane >> 4) < left)
                    d.q[s] = *reinterpret_cast<const v4i*>(q + (int64_t(t) * 128 + s * 64) + at);
            }
        }
    }
};

// Rows of the other operand, bf16, of which there are at most 16 / P at a time.
// With few of them most of an operand's 16 places would stay empty, and every
// load instruction takes the same time however few bytes are new in it; so lane
// (i, g) loads for row i % (16 / P), and for product i / (16 / P) of P in turn, and
// one load serves P products. Each of those has sums of its own, of which the 16
// / P columns are valid that hold its own elements. The second kernel, whose rows
// come twice, packs up to 2 slots fourfold and up to 4 twofold; the first, with four
// blocks of weights per load of rows, does not (its registers spill). Measured on
// MI355X, both kernels, packed and not, us: 256 experts of 7168 -> 2048, 4 bits, 4
// tokens 119 and 123, 16 tokens 356 and 371, 64 tokens 825 and 847; 64 of 2048 ->
// 1408, 8 tokens 50.4 and 55.7 (bf16 137 and 143); 32 of 256 -> 128, 16 tokens 15.6
// and 15.0.
template <bool FOUR, int P>
struct Rows {
    static constexpr int kRows = 16 / P;
    static constexpr int kLoads = Step<FOUR>::kProducts / P;
    // Byte of lane (i, g)'s elements in a step's first load.
    static __device__ uint32_t within(int i, int g) { return (i / kRows) * 64 + g * 16; }
    static __device__ __forceinline__ void load(const char* base, int32_t t, uint32_t at,
                                                v4i (&d)[kLoads]) {
        reform(at);
#pragma unroll
        for (int j = 0; j < kLoads; ++j)
            d[j] = *reinterpret_cast<const v4i*>(
                base + (int64_t(t) * (Step<FOUR>::kElems * 2) + j * P * 64) + at);
    }
    // The last step of a sum that ends inside it, `left` 8-element chunks.
    static __device__ __forceinline__ void load_last(const char* base, int32_t t, int left,
                                                     uint32_t at, int i, int g, v4i (&d)[kLoads]) {
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            d[j] = v4i{0, 0, 0, 0};
            if ((j * P + i / kRows) * 4 + g < left)
                d[j] = *reinterpret_cast<const v4i*>(
                    base + (int64_t(t) * (Step<FOUR>::kElems * 2) + j * P * 64) + at);
        }
    }
};
// The P sums of a block joined: lane (i, g) gets row i % (16 / P)'s.
template <int P>
__device__ __forceinline__ f32x4 join_products(const f32x4 (&acc)[P], int lane) {
    constexpr int R = 16 / P;
    f32x4 v = acc[0];
    if constexpr (P > 1) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float sum = 0.0f;
#pragma unroll
            for (int q = 0; q < P; ++q)
                sum += __shfl(acc[q][k], (lane & 48) + q * R + (lane & (R - 1)), 64);
            v[k] = sum;
        }
    }
    return v;
}

// The experts in use, in ascending order (found by a bit per expert). Every
// thread of the workgroup calls it; `ids` are read once.
struct InUse {
    uint32_t bits[kMaxWords];
    int32_t count;
    int16_t expert[kMaxLayerSlots];
    int16_t id[kMaxLayerSlots];         // of each slot, -1 for none
};
__device__ inline void find_in_use(InUse& u, const int32_t* ids, int slots, int32_t E) {
    const int lane = threadIdx.x & 63;
    if (threadIdx.x < kMaxWords) u.bits[threadIdx.x] = 0;
    __syncthreads();
    for (int p = threadIdx.x; p < slots; p += blockDim.x) {
        const int32_t e = ids[p];
        const bool some = e >= 0 && e < E;
        if (some) atomicOr(&u.bits[e >> 5], 1u << (e & 31));
        u.id[p] = static_cast<int16_t>(some ? e : -1);
    }
    __syncthreads();
    if (threadIdx.x < 64) {
        uint32_t word = lane < kMaxWords ? u.bits[lane] : 0;
        const int mine = __popc(word);
        int incl = mine;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int v = __shfl_up(incl, d, 64);
            if (lane >= d) incl += v;
        }
        int at = incl - mine;
        while (word) {
            u.expert[at++] = static_cast<int16_t>(lane * 32 + __ffs(word) - 1);
            word &= word - 1;
        }
        if (lane == 63) u.count = incl;
    }
    __syncthreads();
}

// Slots of expert e, ascending, into `list`; their number and that of the slots
// of lower experts. A wavefront calls it by itself.
struct Found {
    int n, before;
};
__device__ inline Found find_slots(int16_t* list, const InUse& u, int slots, int32_t e) {
    const int lane = threadIdx.x & 63;
    Found f = {0, 0};
    for (int p0 = 0; p0 < slots; p0 += 64) {
        const int p = p0 + lane;
        const int32_t id = p < slots ? u.id[p] : -1;
        const uint64_t all = __ballot(id == e);
        if (id == e)
            list[f.n + __popcll(all & ((uint64_t(1) << lane) - 1))] = static_cast<int16_t>(p);
        f.n += __popcll(all);
        f.before += __popcll(__ballot(id >= 0 && id < e));
    }
    return f;
}
// Between a wavefront's own LDS writes and reads by its other lanes.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Where h keeps the 32 elements of group `group` of row `row` (their rests lie 64
// bytes behind them).
template <bool FOUR>
__device__ __forceinline__ int64_t h_at(int32_t slots, int32_t row, int32_t group) {
    constexpr int kGroups = Step<FOUR>::kProducts;
    return ((int64_t(group / kGroups) * slots + row) * kGroups + group % kGroups) * 128;
}

// ---- Gate and up projections, the activation and the product ----------------

constexpr int gate_waves(bool four) { return four ? 4 : 8; }
constexpr int kGateBlocks = 4;          // two of gate rows, two of up rows

template <bool FOUR, bool WIDE>
__global__ __launch_bounds__(gate_waves(FOUR) * 64, WIDE ? 2 : 4)
void few_tokens_gate_kernel(const char* __restrict__ x, const int32_t* __restrict__ ids, int32_t T,
                            int32_t K, int32_t E, const char* __restrict__ w,
                            const char* __restrict__ scales, int32_t D, int32_t F, int32_t ftiles,
                            int32_t act, char* __restrict__ h) {
    typedef Step<FOUR> S;
    constexpr int kWaves = gate_waves(FOUR);
    __shared__ InUse in_use;
    __shared__ int16_t list[kMaxLayerSlots];
    __shared__ Found found;
    __shared__ f32x4 part[kWaves][kGateBlocks][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int slots = T * K;
    const int32_t which = blockIdx.x / ftiles, ft = blockIdx.x % ftiles;
    find_in_use(in_use, ids, slots, E);
    if (which >= in_use.count) return;
    const int32_t e = __builtin_amdgcn_readfirstlane(in_use.expert[which]);
    if (wave == 0) {
        const Found f = find_slots(list, in_use, slots, e);
        if (lane == 0) found = f;
    }
    __syncthreads();
    const int n = __builtin_amdgcn_readfirstlane(found.n);
    const int row0 = __builtin_amdgcn_readfirstlane(found.before);
    const int i = lane & 15, g = lane >> 4;
    const int32_t f0 = ft * 32;
    const int32_t steps = (D + S::kElems - 1) / S::kElems;
    const int32_t full = D / S::kElems;

    // Blocks past the matrix read its last rows and are not stored.
    Block<FOUR> blocks[kGateBlocks];
    uint32_t at[kGateBlocks];
#pragma unroll
    for (int b = 0; b < kGateBlocks; ++b) {
        const bool up = b >= 2;
        const int32_t nb = (F + 15) / 16;
        const int32_t ob = min(f0 / 16 + b % 2, nb - 1);
        if constexpr (FOUR) {
            const int64_t blk = int64_t(e) * nb * 2 + (up ? nb : 0) + ob;
            blocks[b].q = w + blk * steps * 1024;
        } else {
            blocks[b].q = w + (int64_t(e) * F * 2 + (up ? F : 0) + ob * 16) * (int64_t(D) * 2);
        }
        at[b] = Block<FOUR>::offset(lane, min(i, F - 1 - ob * 16), int64_t(D) * 2);
    }
    // Lane group g loads the scales of block g.
    const char* scale = scales;
    if constexpr (FOUR) {
        const int32_t nb = (F + 15) / 16;
        const int64_t blk =
            int64_t(e) * nb * 2 + (g >= 2 ? nb : 0) + min(f0 / 16 + g % 2, nb - 1);
        scale += blk * steps * 64 + i * 4;
    }

    // 16 NB / P of the slots from `first` on, or what is left.
    auto run = [&](auto products, auto tiles, int first) {
        constexpr int P = decltype(products)::value, NB = decltype(tiles)::value;
        typedef Rows<FOUR, P> R;
        uint32_t xr[NB];                // below 2^32: 512 rows of at most 2^23 bytes
#pragma unroll
        for (int b = 0; b < NB; ++b)
            xr[b] = static_cast<uint32_t>(list[min(first + b * 16 + i % R::kRows, n - 1)] / K) *
                        (static_cast<uint32_t>(D) * 2) + R::within(i, g);
        struct Data {
            Weights<FOUR> w[kGateBlocks];
            uint32_t scale;
            v4i x[NB][R::kLoads];
        };
        auto load_scale = [&](int32_t t, Data& d) {
            d.scale = 0;
            if constexpr (FOUR)
                d.scale = *reinterpret_cast<const uint32_t*>(scale + int64_t(t) * 64);
        };
        auto load = [&](int32_t t, Data& d) {
            load_scale(t, d);
#pragma unroll
            for (int b = 0; b < NB; ++b) R::load(x, t, xr[b], d.x[b]);
#pragma unroll
            for (int b = 0; b < kGateBlocks; ++b) blocks[b].load(t, at[b], lane, d.w[b]);
            __builtin_amdgcn_sched_barrier(0);
        };
        f32x4 acc[kGateBlocks][NB][P];
#pragma unroll
        for (int a = 0; a < kGateBlocks; ++a)
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int q = 0; q < P; ++q) acc[a][b][q] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        auto compute = [&](const Data& d) {
            uint32_t sc[kGateBlocks];
            spread(d.scale, sc);
#pragma unroll
            for (int s = 0; s < S::kProducts; ++s)
#pragma unroll
                for (int a = 0; a < kGateBlocks; ++a) {
                    const bf16x8 fw = d.w[a].frag(s, sc[a]);
#pragma unroll
                    for (int b = 0; b < NB; ++b)
                        acc[a][b][s % P] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            fw, __builtin_bit_cast(bf16x8, d.x[b][s / P]), acc[a][b][s % P], 0, 0,
                            0);
                }
        };
        Data even, odd;
        int32_t t = wave;
        if (t < full) load(t, even);
        if (t + kWaves < full) load(t + kWaves, odd);
        while (t < full) {
            compute(even);
            if (t + 2 * kWaves < full) load(t + 2 * kWaves, even);
            t += kWaves;
            if (t >= full) break;
            compute(odd);
            if (t + 2 * kWaves < full) load(t + 2 * kWaves, odd);
            t += kWaves;
        }
        if (full < steps && wave == full % kWaves) {
            const int left = (D - full * S::kElems) / 8;
#pragma unroll
            for (int b = 0; b < NB; ++b) R::load_last(x, full, left, xr[b], i, g, even.x[b]);
            load_scale(full, even);
#pragma unroll
            for (int b = 0; b < kGateBlocks; ++b)
                blocks[b].load_last(full, left, at[b], lane, even.w[b]);
            compute(even);
        }

        // Join the wavefronts' sums, in wavefront order.
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            __syncthreads();
#pragma unroll
            for (int a = 0; a < kGateBlocks; ++a)
                part[wave][a][lane] = join_products<P>(acc[a][b], lane);
            __syncthreads();
            if (wave < 2) {
                f32x4 v = part[0][wave][lane], u = part[0][wave + 2][lane];
#pragma unroll
                for (int p = 1; p < kWaves; ++p) {
                    v += part[p][wave][lane];
                    u += part[p][wave + 2][lane];
                }
                const int r = first + b * 16 + i;
                const int32_t f = f0 + wave * 16 + g * 4;
                if (i < R::kRows && r < n && f < F) {
                    f32x4 rest;
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[k] = activate(act, v[k]) * u[k];
                    const v2i high = pack_bf16x4(v);
                    // What the rounding left; nothing where that is not a number.
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t half = static_cast<uint32_t>(high[k >> 1]);
                        const float back =
                            __uint_as_float(k & 1 ? half & 0xFFFF0000u : half << 16);
                        rest[k] = fabsf(back) < INFINITY ? v[k] - back : 0.0f;
                    }
                    char* to = h + h_at<FOUR>(slots, row0 + r, f / 32) + f % 32 * 2;
                    *reinterpret_cast<v2i*>(to) = high;
                    *reinterpret_cast<v2i*>(to + 64) = pack_bf16x4(rest);
                }
            }
        }
    };
    const std::integral_constant<int, 1> one;
    for (int first = 0; first < n; first += WIDE ? 32 : 16)
        run(one, std::integral_constant<int, WIDE ? 2 : 1>{}, first);
}

// ---- Down projection and the sum over the slots ------------------------------

constexpr int kDownWaves = 8;

// Parts that the second kernel splits each expert's sum into, at most: what a
// workgroup's LDS holds of their results.
int most_parts(int slots) { return slots <= 64 ? 8 : slots <= 128 ? 4 : slots <= 256 ? 2 : 1; }

template <bool FOUR, bool WIDE, int CB>
__global__ __launch_bounds__(kDownWaves * 64, CB == 1 ? 4 : 2)
void few_tokens_down_kernel(const char* __restrict__ h, const int32_t* __restrict__ ids,
                            const float* __restrict__ scores, int32_t T, int32_t K, int32_t E,
                            const char* __restrict__ w, const char* __restrict__ scales, int32_t D,
                            int32_t F, int32_t most, __bf16* __restrict__ y) {
    typedef Step<FOUR> S;
    extern __shared__ f32x4 results[];          // [part][slot][chunks of 4 columns]
    __shared__ InUse in_use;
    __shared__ int16_t lists[kDownWaves][kMaxLayerSlots];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int slots = T * K;
    constexpr int kColumns = 16 * CB;
    const int32_t c0 = blockIdx.x * kColumns;
    find_in_use(in_use, ids, slots, E);
    const int count = __builtin_amdgcn_readfirstlane(in_use.count);
    const int i = lane & 15, g = lane >> 4;
    const int32_t steps = (F + S::kElems - 1) / S::kElems;
    const int32_t full = F / S::kElems;
    // The fewest parts that keep the wavefronts busy alike.
    int parts = 1;
    while (parts < most && parts * 2 <= steps &&
           (count * parts + kDownWaves - 1) / kDownWaves * kDownWaves * 8 > count * parts * 9)
        parts *= 2;

    for (int task = wave; task < count * parts; task += kDownWaves) {
        const int32_t e = __builtin_amdgcn_readfirstlane(in_use.expert[task / parts]);
        const int piece = task % parts;
        const int32_t from = static_cast<int32_t>(int64_t(steps) * piece / parts);
        const int32_t to = static_cast<int32_t>(int64_t(steps) * (piece + 1) / parts);
        int16_t* list = lists[wave];
        wave_sync();                // the last task's reads of it are done
        const Found f = find_slots(list, in_use, slots, e);
        wave_sync();
        const int n = f.n;
        // Blocks past the matrix read its last rows and are not stored.
        Block<FOUR> blocks[CB];
        const char* scale[CB];
        uint32_t at[CB];
#pragma unroll
        for (int c = 0; c < CB; ++c) {
            const int32_t nb = (D + 15) / 16;
            const int32_t ob = min(c0 / 16 + c, nb - 1);
            scale[c] = scales;
            if constexpr (FOUR) {
                const int64_t blk = int64_t(e) * nb + ob;
                blocks[c].q = w + blk * steps * 1024;
                scale[c] += blk * steps * 64;
            } else {
                blocks[c].q = w + (int64_t(e) * D + ob * 16) * (int64_t(F) * 2);
            }
            at[c] = Block<FOUR>::offset(lane, min(i, D - 1 - ob * 16), int64_t(F) * 2);
        }
        // 8 NB / P of the slots from `first` on, or what is left: the first half of
        // the rows are h's rounded numbers, the second what the rounding left.
        auto run = [&](auto products, auto tiles, int first) {
            constexpr int P = decltype(products)::value, NB = decltype(tiles)::value;
            typedef Rows<FOUR, P> R;
            constexpr int kSlots = R::kRows / 2;
            // Rows of h: the slots in the order of their experts. A step's rows
            // lie together, 128 bytes for each group of 32 elements.
            constexpr int kRowBytes = S::kProducts * 128;
            const char* hb = h + int64_t(f.before + first) * kRowBytes;
            const int64_t pitch = int64_t(slots) * kRowBytes;
            uint32_t hr[NB];
#pragma unroll
            for (int b = 0; b < NB; ++b)
                hr[b] = min(b * 8 + i % kSlots, n - first - 1) * kRowBytes +
                        i / R::kRows * 128 + (i % R::kRows < kSlots ? 0 : 64) + g * 16;
            struct Data {
                Weights<FOUR> w[CB];
                v4i x[NB][R::kLoads];
            };
            auto load = [&](int32_t t, Data& d) {
#pragma unroll
                for (int c = 0; c < CB; ++c) blocks[c].load(t, at[c], lane, d.w[c]);
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    uint32_t from = hr[b];
                    reform(from);
#pragma unroll
                    for (int j = 0; j < R::kLoads; ++j)
                        d.x[b][j] = *reinterpret_cast<const v4i*>(
                            hb + (int64_t(t) * pitch + j * P * 128) + from);
                }
                __builtin_amdgcn_sched_barrier(0);
            };
            // The scales of 4 steps, lane group g's of step t + g.
            auto load_scales = [&](int32_t t, uint32_t (&d)[CB]) {
                const uint32_t so = min(t + g, steps - 1) * 64 + i * 4;
#pragma unroll
                for (int c = 0; c < CB; ++c)
                    d[c] = FOUR ? *reinterpret_cast<const uint32_t*>(scale[c] + so) : 0;
            };
            f32x4 acc[CB][NB][P];
#pragma unroll
            for (int c = 0; c < CB; ++c)
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int q = 0; q < P; ++q) acc[c][b][q] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            uint32_t next[CB], sc[CB][4];
            auto spread_scales = [&] {
#pragma unroll
                for (int c = 0; c < CB; ++c) spread(next[c], sc[c]);
            };
            auto compute = [&](const Data& d, int j) {
#pragma unroll
                for (int s = 0; s < S::kProducts; ++s)
#pragma unroll
                    for (int c = 0; c < CB; ++c) {
                        const bf16x8 fw = d.w[c].frag(s, sc[c][j]);
#pragma unroll
                        for (int b = 0; b < NB; ++b)
                            acc[c][b][s % P] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                fw, __builtin_bit_cast(bf16x8, d.x[b][s / P]), acc[c][b][s % P], 0,
                                0, 0);
                    }
            };
            const int32_t end = min(to, full);
            // `kDepth` steps in flight, the scales of 4 at a time.
            constexpr int kDepth = NB == 1 ? 4 : 2;
            Data ring[kDepth];
            load_scales(from, next);
#pragma unroll
            for (int j = 0; j < kDepth; ++j)
                if (from + j < end) load(from + j, ring[j]);
            for (int32_t t = from; t < end;) {
                spread_scales();
                if (t + 4 < steps) load_scales(t + 4, next);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (t >= end) break;
                    compute(ring[j % kDepth], j);
                    if (t + kDepth < end) load(t + kDepth, ring[j % kDepth]);
                    ++t;
                }
            }
            if (full < to) {
                const int left = (F - full * S::kElems) / 8;
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int j = 0; j < R::kLoads; ++j) {
                        ring[0].x[b][j] = v4i{0, 0, 0, 0};
                        if ((j * P + i / R::kRows) * 4 + g < left)
                            ring[0].x[b][j] = *reinterpret_cast<const v4i*>(
                                hb + (int64_t(full) * pitch + j * P * 128) + hr[b]);
                    }
#pragma unroll
                for (int c = 0; c < CB; ++c)
                    blocks[c].load_last(full, left, at[c], lane, ring[0].w[c]);
                load_scales(full, next);
                spread_scales();
                compute(ring[0], 0);
            }
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int c = 0; c < CB; ++c) {
                    f32x4 v = join_products<P>(acc[c][b], lane);
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[k] += __shfl_xor(v[k], kSlots, 64);
                    const int r = first + b * 8 + i;
                    if (i < kSlots && r < n)
                        results[((piece * slots + list[r]) * CB + c) * 4 + g] = v;
                }
        };
        const std::integral_constant<int, 1> one;
        for (int first = 0; first < n;) {
            const int left = n - first;
            if (FOUR && left <= 2) {
                run(std::integral_constant<int, S::kProducts>{}, one, first);
                first += 2;
            } else if (left <= 4) {
                run(std::integral_constant<int, 2>{}, one, first);
                first += 4;
            } else {
                run(one, std::integral_constant<int, WIDE ? 2 : 1>{}, first);
                first += WIDE ? 16 : 8;
            }
        }
    }
    __syncthreads();
    const float* sums = reinterpret_cast<const float*>(results);
    for (int q = threadIdx.x; q < T * kColumns; q += kDownWaves * 64) {
        const int t = q / kColumns, c = q % kColumns;
        if (c0 + c >= D) continue;
        float v = 0.0f;
        for (int k = 0; k < K; ++k) {
            const int p = t * K + k;
            const int32_t e = ids[p];
            if (e < 0 || e >= E) continue;
            float one = sums[p * kColumns + c];
            for (int j = 1; j < parts; ++j) one += sums[(j * slots + p) * kColumns + c];
            v = __builtin_fmaf(scores[p], one, v);
        }
        y[int64_t(t) * D + c0 + c] = static_cast<__bf16>(v);
    }
}

int64_t gate_tiles(const LayerArgs& a) { return (int64_t(a.F) + 31) / 32; }
int64_t gate_workgroups(const LayerArgs& a) {
    const int64_t slots = int64_t(a.T) * a.K;
    return gate_tiles(a) * (slots < a.E ? slots : a.E);
}

template <bool FOUR, bool WIDE>
hipError_t launch(const LayerArgs& a, hipStream_t stream) {
    const char* w1 = static_cast<const char*>(a.w_gate_up);
    const char* w2 = static_cast<const char*>(a.w_down);
    const int slots = a.T * a.K;
    hipLaunchKernelGGL((few_tokens_gate_kernel<FOUR, WIDE>),
                       dim3(static_cast<uint32_t>(gate_workgroups(a))), dim3(gate_waves(FOUR) * 64),
                       0, stream, static_cast<const char*>(a.x), a.ids, a.T, a.K, a.E, w1,
                       w1 + mxfp4_tiles(a.E, 2 * a.F, a.D) * 1024, a.D, a.F,
                       static_cast<int32_t>(gate_tiles(a)), a.activation,
                       static_cast<char*>(a.workspace));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int most = most_parts(slots);
    auto down = few_tokens_down_kernel<FOUR, WIDE, 1>;
    // 16 columns of y per workgroup, or 32 where 16 give every CU more than one: every
    // row of h then serves twice the weights. Measured on MI355X, 16 and 32, us: 256
    // experts of 7168 -> 2048, 4 bits, 1 token 40.1 and 40.3, 64 tokens 881 and 825; 8 of
    // 4096 -> 4096, 8 tokens 43.9 and 48.4 (bf16 154 and 175); 64 of 2048 -> 1408, 32
    // tokens 85 and 100 (239 and 312).
    int columns = 16;
    if (a.D > 16 * 256) {
        down = few_tokens_down_kernel<FOUR, WIDE, 2>;
        columns = 32;
    }
    hipLaunchKernelGGL(down, dim3(static_cast<uint32_t>((a.D + columns - 1) / columns)),
                       dim3(kDownWaves * 64), slots * most * 4 * columns, stream,
                       static_cast<const char*>(a.workspace), a.ids, a.scores, a.T, a.K, a.E, w2,
                       w2 + mxfp4_tiles(a.E, a.D, a.F) * 1024, a.D, a.F, most,
                       static_cast<__bf16*>(a.y));
    return hipGetLastError();
}

}  // namespace

int64_t few_tokens_grid(const LayerArgs& a) { return gate_workgroups(a) * (gate_waves(a.four) * 64); }

hipError_t launch_few_tokens(const LayerArgs& a, hipStream_t stream) {
    // Twice the slots per pass over the weights where experts have many: fewer passes,
    // but half the wavefronts per CU and twice the products of a pass that has few.
    // Measured on MI355X, both kernels, one against two times 16 (8) slots, us: 8 experts
    // of 4096 -> 4096 at 4 slots each 170 and 175 (4 bits 51 and 59), at 8 194 and 189
    // (69 and 74), at 16 286 and 230 (115 and 110); 64 of 2048 -> 1408 at 6 each 292 and
    // 331 (121 and 149).
    if (int64_t(a.T) * a.K >= int64_t(12) * a.E)
        return a.four ? launch<true, true>(a, stream) : launch<false, true>(a, stream);
    return a.four ? launch<true, false>(a, stream) : launch<false, false>(a, stream);
}

}  // namespace moe
