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
// rounding that a bf16 h would bring costs nothing to avoid.
//
// Bound: the bytes of the weights in use, read once each, straight into the
// registers the matrix cores read.
#include "expert_kernels.h"
#include "expert_mma.h"
#include "expert_mxfp4.h"
#include "layer_kernels.h"

namespace moe {
namespace {

constexpr int kMaxWords = 32;           // of a bit per expert (1024)

// What a step of the sum takes from memory for one 16-feature block.
template <bool FOUR>
struct Weights;
template <>
struct Weights<true> : Mxfp4Step {};
template <>
struct Weights<false> {
    v4i q[2];
    __device__ bf16x8 frag(int s) const { return __builtin_bit_cast(bf16x8, q[s]); }
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
    const char* scale;
    // Lane (i, g)'s offsets, the same for all blocks of a kernel but for a
    // clamped row.
    static __device__ uint32_t offset(int lane, int32_t row, int64_t pitch) {
        return FOUR ? lane * 16 : static_cast<uint32_t>(row * pitch) + (lane >> 4) * 16;
    }
    __device__ __forceinline__ void load(int32_t t, uint32_t at, int lane, Weights<FOUR>& d) const {
        if constexpr (FOUR) {
            uint32_t so = (lane & 15) * 4;
            reform(at);
            reform(so);
            d.q = __builtin_nontemporal_load(
                reinterpret_cast<const v4i*>(q + int64_t(t) * 1024 + at));
            d.scale = *reinterpret_cast<const uint32_t*>(scale + int64_t(t) * 64 + so);
        } else {
            reform(at);
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

// Rows of the other operand, bf16: 8 elements of this lane's row (offset `at` from
// the uniform `base`) for each product of step t.
template <bool FOUR>
__device__ __forceinline__ void load_rows(const char* base, int32_t t, uint32_t at,
                                          v4i (&d)[Step<FOUR>::kProducts]) {
    reform(at);
#pragma unroll
    for (int s = 0; s < Step<FOUR>::kProducts; ++s)
        d[s] = *reinterpret_cast<const v4i*>(base + (int64_t(t) * (Step<FOUR>::kElems * 2) + s * 64) +
                                             at);
}
template <bool FOUR>
__device__ __forceinline__ void load_rows_last(const char* base, int32_t t, int left, uint32_t at,
                                               int lane, v4i (&d)[Step<FOUR>::kProducts]) {
#pragma unroll
    for (int s = 0; s < Step<FOUR>::kProducts; ++s) {
        d[s] = v4i{0, 0, 0, 0};
        if (4 * s + (lane >> 4) < left)
            d[s] = *reinterpret_cast<const v4i*>(
                base + (int64_t(t) * (Step<FOUR>::kElems * 2) + s * 64) + at);
    }
}

// The experts in use, in ascending order, from the slots' ids (a bit per expert
// first). Every thread of the workgroup calls it.
struct InUse {
    uint32_t bits[kMaxWords];
    int16_t expert[kMaxLayerSlots];
    int32_t count;
};
__device__ inline void find_in_use(InUse& u, const int32_t* ids, int slots, int32_t E) {
    if (threadIdx.x < kMaxWords) u.bits[threadIdx.x] = 0;
    __syncthreads();
    for (int p = threadIdx.x; p < slots; p += blockDim.x) {
        const int32_t e = ids[p];
        if (e >= 0 && e < E) atomicOr(&u.bits[e >> 5], 1u << (e & 31));
    }
    __syncthreads();
    if (threadIdx.x < 64) {
        const int lane = threadIdx.x;
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

// Slots of expert e, ascending, into `list`; their number. A wavefront calls
// it by itself.
__device__ inline int find_slots(int16_t* list, const int32_t* ids, int slots, int32_t e) {
    const int lane = threadIdx.x & 63;
    int n = 0;
    for (int p0 = 0; p0 < slots; p0 += 64) {
        const int p = p0 + lane;
        const bool mine = p < slots && ids[p] == e;
        const uint64_t all = __ballot(mine);
        if (mine) list[n + __popcll(all & ((uint64_t(1) << lane) - 1))] = static_cast<int16_t>(p);
        n += __popcll(all);
    }
    return n;
}
// Between a wavefront's own LDS writes and reads by its other lanes.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// ---- Gate and up projections, the activation and the product ----------------

constexpr int gate_waves(bool four) { return four ? 4 : 8; }
constexpr int kGateBlocks = 4;          // two of gate rows, two of up rows

template <bool FOUR, int NB>
__global__ __launch_bounds__(gate_waves(FOUR) * 64, NB == 1 ? 4 : 2)
void few_tokens_gate_kernel(const char* __restrict__ x, const int32_t* __restrict__ ids, int32_t T,
                            int32_t K, int32_t E, const char* __restrict__ w,
                            const char* __restrict__ scales, int32_t D, int32_t F, int32_t ftiles,
                            int32_t act, char* __restrict__ h) {
    typedef Step<FOUR> S;
    constexpr int kWaves = gate_waves(FOUR);
    __shared__ InUse in_use;
    __shared__ int16_t list[kMaxLayerSlots];
    __shared__ int32_t list_size;
    __shared__ f32x4 part[kWaves][kGateBlocks][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int slots = T * K;
    const int32_t which = blockIdx.x / ftiles, ft = blockIdx.x % ftiles;
    find_in_use(in_use, ids, slots, E);
    if (which >= in_use.count) return;
    const int32_t e = __builtin_amdgcn_readfirstlane(in_use.expert[which]);
    if (wave == 0) {
        const int n = find_slots(list, ids, slots, e);
        if (lane == 0) list_size = n;
    }
    __syncthreads();
    const int n = __builtin_amdgcn_readfirstlane(list_size);
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
            blocks[b].scale = scales + blk * steps * 64;
        } else {
            blocks[b].q = w + (int64_t(e) * F * 2 + (up ? F : 0) + ob * 16) * (int64_t(D) * 2);
            blocks[b].scale = nullptr;
        }
        at[b] = Block<FOUR>::offset(lane, min(i, F - 1 - ob * 16), int64_t(D) * 2);
    }

    // 16 NB of the slots, or what is left.
    for (int first = 0; first < n; first += 16 * NB) {
        uint32_t xr[NB];                // below 2^32: 512 rows of at most 2^23 bytes
#pragma unroll
        for (int b = 0; b < NB; ++b)
            xr[b] = static_cast<uint32_t>(list[min(first + b * 16 + i, n - 1)] / K) *
                        (static_cast<uint32_t>(D) * 2) + g * 16;
        struct Data {
            Weights<FOUR> w[kGateBlocks];
            v4i x[NB][S::kProducts];
        };
        auto load = [&](int32_t t, Data& d) {
#pragma unroll
            for (int b = 0; b < NB; ++b) load_rows<FOUR>(x, t, xr[b], d.x[b]);
#pragma unroll
            for (int b = 0; b < kGateBlocks; ++b) blocks[b].load(t, at[b], lane, d.w[b]);
            __builtin_amdgcn_sched_barrier(0);
        };
        f32x4 acc[kGateBlocks][NB];
#pragma unroll
        for (int a = 0; a < kGateBlocks; ++a)
#pragma unroll
            for (int b = 0; b < NB; ++b) acc[a][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        auto compute = [&](const Data& d) {
#pragma unroll
            for (int s = 0; s < S::kProducts; ++s)
#pragma unroll
                for (int a = 0; a < kGateBlocks; ++a) {
                    const bf16x8 fw = d.w[a].frag(s);
#pragma unroll
                    for (int b = 0; b < NB; ++b)
                        acc[a][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            fw, __builtin_bit_cast(bf16x8, d.x[b][s]), acc[a][b], 0, 0, 0);
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
            for (int b = 0; b < NB; ++b) load_rows_last<FOUR>(x, full, left, xr[b], lane, even.x[b]);
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
            for (int a = 0; a < kGateBlocks; ++a) part[wave][a][lane] = acc[a][b];
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
                if (r < n && f < F) {
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
                    char* at = h + (int64_t(list[r]) * F + f) * 2;
                    *reinterpret_cast<v2i*>(at) = high;
                    *reinterpret_cast<v2i*>(at + int64_t(slots) * F * 2) = pack_bf16x4(rest);
                }
            }
        }
    }
}

// ---- Down projection and the sum over the slots ------------------------------

constexpr int kDownWaves = 8;

// Parts that the second kernel splits each expert's sum into, at most: what a
// workgroup's LDS holds of their results.
int most_parts(int slots) { return slots <= 64 ? 8 : slots <= 128 ? 4 : slots <= 256 ? 2 : 1; }

template <bool FOUR, int NB>
__global__ __launch_bounds__(kDownWaves * 64, 4)
void few_tokens_down_kernel(const char* __restrict__ h, const int32_t* __restrict__ ids,
                            const float* __restrict__ scores, int32_t T, int32_t K, int32_t E,
                            const char* __restrict__ w, const char* __restrict__ scales, int32_t D,
                            int32_t F, int32_t most, __bf16* __restrict__ y) {
    typedef Step<FOUR> S;
    extern __shared__ f32x4 results[];          // [part][slot][4 chunks of 4 columns]
    __shared__ InUse in_use;
    __shared__ int16_t lists[kDownWaves][kMaxLayerSlots];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int slots = T * K;
    const int32_t c0 = blockIdx.x * 16;
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
        const int n = find_slots(list, ids, slots, e);
        wave_sync();
        Block<FOUR> block;
        if constexpr (FOUR) {
            const int64_t blk = int64_t(e) * ((D + 15) / 16) + c0 / 16;
            block.q = w + blk * steps * 1024;
            block.scale = scales + blk * steps * 64;
        } else {
            block.q = w + (int64_t(e) * D + c0) * (int64_t(F) * 2);
            block.scale = nullptr;
        }
        const uint32_t at = Block<FOUR>::offset(lane, min(i, D - 1 - c0), int64_t(F) * 2);
        // 8 NB of the slots, or what is left; lanes i < 8 take h's rounded
        // numbers, the others what the rounding left.
        for (int first = 0; first < n; first += 8 * NB) {
            uint32_t hr[NB];            // below 2^32: 1024 rows of at most 2^22 bytes
#pragma unroll
            for (int b = 0; b < NB; ++b)
                hr[b] = static_cast<uint32_t>(list[min(first + b * 8 + (i & 7), n - 1)] +
                                              (i < 8 ? 0 : slots)) *
                            (static_cast<uint32_t>(F) * 2) + g * 16;
            struct Data {
                Weights<FOUR> w;
                v4i x[NB][S::kProducts];
            };
            auto load = [&](int32_t t, Data& d) {
                block.load(t, at, lane, d.w);
#pragma unroll
                for (int b = 0; b < NB; ++b) load_rows<FOUR>(h, t, hr[b], d.x[b]);
                __builtin_amdgcn_sched_barrier(0);
            };
            f32x4 acc[NB];
#pragma unroll
            for (int b = 0; b < NB; ++b) acc[b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            auto compute = [&](const Data& d) {
#pragma unroll
                for (int s = 0; s < S::kProducts; ++s) {
                    const bf16x8 fw = d.w.frag(s);
#pragma unroll
                    for (int b = 0; b < NB; ++b)
                        acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            fw, __builtin_bit_cast(bf16x8, d.x[b][s]), acc[b], 0, 0, 0);
                }
            };
            const int32_t end = min(to, full);
            Data even, odd;
            int32_t t = from;
            if (t < end) load(t, even);
            if (t + 1 < end) load(t + 1, odd);
            while (t < end) {
                compute(even);
                if (t + 2 < end) load(t + 2, even);
                if (++t >= end) break;
                compute(odd);
                if (t + 2 < end) load(t + 2, odd);
                ++t;
            }
            if (full < to) {
                const int left = (F - full * S::kElems) / 8;
#pragma unroll
                for (int b = 0; b < NB; ++b)
                    load_rows_last<FOUR>(h, full, left, hr[b], lane, even.x[b]);
                block.load_last(full, left, at, lane, even.w);
                compute(even);
            }
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                f32x4 v = acc[b];
#pragma unroll
                for (int k = 0; k < 4; ++k) v[k] += __shfl_xor(v[k], 8, 64);
                const int r = first + b * 8 + i;
                if (i < 8 && r < n) results[(piece * slots + list[r]) * 4 + g] = v;
            }
        }
    }
    __syncthreads();
    const float* sums = reinterpret_cast<const float*>(results);
    for (int q = threadIdx.x; q < T * 16; q += kDownWaves * 64) {
        const int t = q >> 4, c = q & 15;
        if (c0 + c >= D) continue;
        float v = 0.0f;
        for (int k = 0; k < K; ++k) {
            const int p = t * K + k;
            const int32_t e = ids[p];
            if (e < 0 || e >= E) continue;
            float one = sums[p * 16 + c];
            for (int j = 1; j < parts; ++j) one += sums[(j * slots + p) * 16 + c];
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

template <bool FOUR, int NB>
hipError_t launch(const LayerArgs& a, hipStream_t stream) {
    const char* w1 = static_cast<const char*>(a.w_gate_up);
    const char* w2 = static_cast<const char*>(a.w_down);
    const int slots = a.T * a.K;
    hipLaunchKernelGGL((few_tokens_gate_kernel<FOUR, NB>),
                       dim3(static_cast<uint32_t>(gate_workgroups(a))), dim3(gate_waves(FOUR) * 64),
                       0, stream, static_cast<const char*>(a.x), a.ids, a.T, a.K, a.E, w1,
                       w1 + mxfp4_tiles(a.E, 2 * a.F, a.D) * 1024, a.D, a.F,
                       static_cast<int32_t>(gate_tiles(a)), a.activation,
                       static_cast<char*>(a.workspace));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int most = most_parts(slots);
    hipLaunchKernelGGL((few_tokens_down_kernel<FOUR, NB>),
                       dim3(static_cast<uint32_t>((a.D + 15) / 16)), dim3(kDownWaves * 64),
                       slots * most * 64, stream, static_cast<const char*>(a.workspace), a.ids,
                       a.scores, a.T, a.K, a.E, w2, w2 + mxfp4_tiles(a.E, a.D, a.F) * 1024, a.D,
                       a.F, most, static_cast<__bf16*>(a.y));
    return hipGetLastError();
}

}  // namespace

int64_t few_tokens_grid(const LayerArgs& a) { return gate_workgroups(a) * (gate_waves(a.four) * 64); }

hipError_t launch_few_tokens(const LayerArgs& a, hipStream_t stream) {
    // Twice the slots per pass over the weights where experts have many.
    if (int64_t(a.T) * a.K >= int64_t(4) * a.E)
        return a.four ? launch<true, 2>(a, stream) : launch<false, 2>(a, stream);
    return a.four ? launch<true, 1>(a, stream) : launch<false, 1>(a, stream);
}

}  // namespace moe
