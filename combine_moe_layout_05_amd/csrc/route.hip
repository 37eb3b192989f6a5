// The router on gfx950: the K experts of every token and their scores from the
// router's logits, and the gradient of the logits.
//
// With l the logits of a token, the experts taking part being those whose l is
// neither NaN nor -inf:
//   softmax   p = exp(l - m) / sum of exp(l - m), m the largest l
//   sigmoid   p = 1 / (1 + exp(-l))
// The K largest of v are chosen, equal ones by index; v is l, which has p's order,
// or with a bias sigmoid(l) + bias. That is computed in 64 bits, so that the order
// of near values is that of the formula and not that of an exponential's last
// digit. With groups of consecutive experts only those of the `kept` best groups
// can be chosen, by the group's largest v (softmax) or the sum of the sigmoids,
// plus their bias, of its two largest (sigmoid), in 64 bits.
//
// Up to 256 experts and 8 of them per token: 16 lanes per token, which select by
// 32-bit keys and check the result, with the slow form for tokens that the check
// does not clear. Else one wavefront per token; lane j holds experts j, j + 64, ...
//
// Bound: for a few tokens a launch, its loads and the chain of the selection (one
// token of 256 experts, 8 groups 4.4 us); for many the vector instructions of the
// selection, not the bytes. Measured on MI355X, 32768 tokens of 256 experts, fp32, 8
// each: softmax 11.5 us (35.7 MB, 3.1 TB/s), sigmoid with bias 14.1, in 8 groups 17.0
// (a wavefront per token 178), in groups without a bias 14.0. A wavefront per token,
// 8192 tokens of 512 experts, 8 each: softmax 15.7, sigmoid 13.5, with bias 24, in 8
// groups 46 and without a bias 40; the gradient 17.2. One token of
// the slow form at the end of a launch costs some 5 us: before groups near the last kept
// and an expert near the last chosen were settled in their lanes, the latter two took
// 18.8 and 22.
#include <cmath>

#include "expert_kernels.h"
#include "layer_kernels.h"

namespace moe {
namespace {

constexpr int kWaves = 4;               // tokens per workgroup

__device__ __forceinline__ float logit_at(const float* p, int64_t i) { return p[i]; }
__device__ __forceinline__ float logit_at(const __bf16* p, int64_t i) {
    return static_cast<float>(p[i]);
}

// Experts that take no part have a logit of -inf from here on.
__device__ __forceinline__ float taking_part(float l) { return l == l ? l : -INFINITY; }

// v moved between lanes by a data-parallel primitive; lanes it gives nothing keep
// theirs.
template <int CTRL, int ROWS>
__device__ __forceinline__ int32_t moved(int32_t v) {
    return __builtin_amdgcn_update_dpp(v, v, CTRL, ROWS, 0xF, false);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ float moved(float v) {
    return __builtin_bit_cast(float, moved<CTRL, ROWS>(__builtin_bit_cast(int32_t, v)));
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double moved(double v) {
    typedef int32_t two __attribute__((ext_vector_type(2)));
    const two w = __builtin_bit_cast(two, v);
    return __builtin_bit_cast(double,
                              two{moved<CTRL, ROWS>(w[0]), moved<CTRL, ROWS>(w[1])});
}
__device__ __forceinline__ float last_lane(float v) {
    return __builtin_bit_cast(
        float, __builtin_amdgcn_readlane(__builtin_bit_cast(int32_t, v), 63));
}
__device__ __forceinline__ double last_lane(double v) {
    typedef int32_t two __attribute__((ext_vector_type(2)));
    const two w = __builtin_bit_cast(two, v);
    return __builtin_bit_cast(double, two{__builtin_amdgcn_readlane(w[0], 63),
                                          __builtin_amdgcn_readlane(w[1], 63)});
}
__device__ __forceinline__ float larger(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ double larger(double a, double b) { return fmax(a, b); }

// The wavefront's largest value (none is a NaN), in every lane: within rows of 16
// by shifts of 1, 2, 4 and 8, then from each row's last lane to the rows behind it.
template <class V>
__device__ __forceinline__ V wave_max(V v) {
    v = larger(v, moved<0x111, 0xF>(v));
    v = larger(v, moved<0x112, 0xF>(v));
    v = larger(v, moved<0x114, 0xF>(v));
    v = larger(v, moved<0x118, 0xF>(v));
    v = larger(v, moved<0x142, 0xA>(v));
    v = larger(v, moved<0x143, 0xC>(v));
    return last_lane(v);
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d, 64);
    return v;
}

// The wavefront's largest of v, and the lowest of the experts that have it.
template <int VALS, class V>
__device__ __forceinline__ void best_of(const V (&v)[VALS], V& top, int& at) {
    top = v[0];
#pragma unroll
    for (int i = 1; i < VALS; ++i) top = larger(top, v[i]);
    top = wave_max(top);
    at = -1;
#pragma unroll
    for (int i = 0; i < VALS; ++i) {
        const uint64_t here = __ballot(v[i] == top);
        if (at < 0 && here) at = i * 64 + __ffsll(static_cast<unsigned long long>(here)) - 1;
    }
}

template <int VALS, class V>
__device__ __forceinline__ void take_out(V (&v)[VALS], int lane, int at) {
#pragma unroll
    for (int i = 0; i < VALS; ++i)
        if (i * 64 + lane == at) v[i] = -INFINITY;
}

__device__ __forceinline__ double sigmoid_64(double l) { return 1.0 / (1.0 + exp(-l)); }
// What a value counts in its group's sum: a logit its sigmoid, others themselves.
__device__ __forceinline__ double in_sum(float l) { return sigmoid_64(l); }
__device__ __forceinline__ double in_sum(double v) { return v; }

// The experts chosen by v (destroyed): lane k gets the k-th, or -1. Groups go by
// their largest value, or, with `pairs`, by the sum of what their two largest count.
template <int VALS, class V>
__device__ int select(V (&v)[VALS], int lane, int K, int E, int groups, int kept, bool pairs) {
    if (groups > 1) {
        const int size = E / groups;
        // Lane g holds group g's value; groups without an expert keep -inf.
        double value = -INFINITY;
        for (int g = 0; g < groups; ++g) {
            V w[VALS];
#pragma unroll
            for (int i = 0; i < VALS; ++i) {
                const int e = i * 64 + lane;
                w[i] = e >= g * size && e < (g + 1) * size ? v[i] : V(-INFINITY);
            }
            V first, second;
            int at;
            best_of<VALS, V>(w, first, at);
            double sum = first;
            if (pairs && first > V(-INFINITY)) {
                sum = in_sum(first);
                take_out<VALS, V>(w, lane, at);
                best_of<VALS, V>(w, second, at);
                if (second > V(-INFINITY)) sum += in_sum(second);
            }
            if (lane == g) value = sum;
        }
        uint64_t open = 0;
        for (int j = 0; j < kept; ++j) {
            const double one[1] = {value};
            double top;
            int at;
            best_of<1, double>(one, top, at);
            if (!(top > -INFINITY)) break;
            open |= uint64_t(1) << at;
            if (lane == at) value = -INFINITY;
        }
#pragma unroll
        for (int i = 0; i < VALS; ++i) {
            const int e = i * 64 + lane;
            if (e < E && !(open >> (e / size) & 1)) v[i] = -INFINITY;
        }
    }
    int mine = -1;
    for (int k = 0; k < K; ++k) {
        V top;
        int at;
        best_of<VALS, V>(v, top, at);
        if (!(top > V(-INFINITY))) break;
        if (lane == k) mine = at;
        take_out<VALS, V>(v, lane, at);
    }
    return mine;
}

// 1 - sigmoid(l) and sigmoid(l), from an exponential that does not overflow: a
// sigmoid below 2^-127 is not lost. The former without the difference, which loses its
// last digits near 1.
__device__ __forceinline__ float sigmoid_rest(float l) {
    const float e = expf(-fabsf(l));
    return (l > 0.0f ? e : 1.0f) / (1.0f + e);
}
__device__ __forceinline__ float sigmoid_32(float l) { return sigmoid_rest(-l); }

// The sigmoids of a token's chosen experts (id >= 0, logit l) and, to renormalize
// them, their sum over its lanes. A sum below 2^-24 is formed again with every sigmoid
// times exp(-top), `top` the largest chosen logit: only the quotients count, and
// numbers near 2^-149 have few digits. Sigmoids that are all 0 in fp32 stay 0.
template <class Max, class Sum>
__device__ __forceinline__ float chosen_sigmoid(int id, float l, bool renormalize, float& sum,
                                                Max max_of, Sum sum_of) {
    float p = id >= 0 ? sigmoid_32(l) : 0.0f;
    if (!renormalize) return p;
    sum = sum_of(p);
    if (sum < 0x1p-24f) {
        const float top = max_of(id >= 0 ? l : -INFINITY);
        const bool some = id >= 0 && top >= -103.972077083991796f;      // 2^-150
        p = some ? expf(l - top) / (1.0f + expf(l)) : 0.0f;
        sum = sum_of(p);
    }
    return p;
}

// The score of a chosen expert in lanes 0 .. K - 1 (id >= 0, logit l), before
// the scale; `top` and `sum` are the softmax's over all experts.
__device__ __forceinline__ float score_of(bool sigmoid, bool renormalize, int id, float l,
                                          float top, float sum) {
    float p = 0.0f;
    if (sigmoid) {
        p = chosen_sigmoid(id, l, renormalize, sum, wave_max<float>, wave_sum);
    } else {
        if (id >= 0) p = expf(l - top);
        if (renormalize) sum = wave_sum(p);
    }
    if (renormalize || !sigmoid) p = sum == 0.0f ? 0.0f : p / sum;
    return p;
}

// The choice of one token by a whole wavefront: lane k < K gets the k-th
// expert or -1. Only experts e with bit e / per of `open` are looked at.
template <int VALS, class L>
__device__ int choose(const L* in, const float* bias, int lane, int32_t K, int32_t E, bool sigmoid,
                      int32_t groups, int32_t kept, uint32_t open = 1, int32_t per = 1024) {
    float l[VALS];
#pragma unroll
    for (int i = 0; i < VALS; ++i) {
        const int e = i * 64 + lane;
        l[i] = e < E && (open >> (e / per) & 1) ? taking_part(logit_at(in, e)) : -INFINITY;
    }
    if (!sigmoid || !bias)
        return select<VALS, float>(l, lane, K, E, groups, kept, sigmoid);
    double v[VALS];
#pragma unroll
    for (int i = 0; i < VALS; ++i) {
        v[i] = -INFINITY;
        if (l[i] > -INFINITY) {
            v[i] = sigmoid_64(l[i]) + static_cast<double>(bias[i * 64 + lane]);
            if (!(v[i] == v[i])) v[i] = -INFINITY;
        }
    }
    return select<VALS, double>(v, lane, K, E, groups, kept, true);
}

template <int VALS, class L>
__global__ __launch_bounds__(kWaves * 64)
void route_kernel(const L* __restrict__ logits, const float* __restrict__ bias, int32_t T,
                  int32_t E, int32_t K, int32_t sigmoid, int32_t renormalize, float scale,
                  int32_t groups, int32_t kept, int32_t* __restrict__ ids,
                  float* __restrict__ scores) {
    const int lane = threadIdx.x & 63;
    const int64_t row = int64_t(blockIdx.x) * (blockDim.x >> 6) + (threadIdx.x >> 6);
    if (row >= T) return;
    const L* in = logits + row * E;
    float top = -INFINITY, sum = 0.0f;
    if (!sigmoid) {
        for (int e = lane; e < E; e += 64) top = fmaxf(top, taking_part(logit_at(in, e)));
        top = wave_max(top);
        if (!renormalize && top > -INFINITY) {
            for (int e = lane; e < E; e += 64) {
                const float v = taking_part(logit_at(in, e));
                if (v > -INFINITY) sum += expf(v - top);
            }
            sum = wave_sum(sum);
        }
    }
    const int id = choose<VALS, L>(in, bias, lane, K, E, sigmoid != 0, groups, kept);
    float p = 0.0f;
    if (id >= 0) p = logit_at(in, id);
    p = score_of(sigmoid, renormalize, id, p, top, sum);
    if (lane < K) {
        ids[row * K + lane] = id;
        scores[row * K + lane] = p * scale;
    }
}

// ---- 16 lanes per token ------------------------------------------------------
//
// Lane j of a token holds up to VALS experts in a row. Each value becomes a
// key of 32 bits: its distance to the token's largest in 24 bits of 2^-20 (16 in
// all), and the expert's index, so that keys differ and equal values go by index.
// A lane sorts its keys, the lanes' lists of 8 are merged by rotations, after which
// all hold the token's 8 largest keys in order: some 60 instructions per token
// where 8 rounds of a search over the wavefront take several hundred.
//
// Then the choice is checked against the values themselves: neighbours in order
// and every other expert below the last, exactly where they are logits, by more
// than the error of a value in 32 bits where they are sigmoids plus a bias.
// Neighbours nearer than that, among them one expert too near to the last, are put
// in order by their values in 64 bits, and so are groups too near to the last kept.
// A token that fails otherwise (two experts too near to the last, three in a group
// too near to each other, fewer experts than slots, values more than 16 apart,
// infinities) is chosen for by the whole wavefront.
constexpr int kLanes = 16;
constexpr int kList = 8;

template <int N>
__device__ __forceinline__ float ror(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int32_t, v),
                                                              0x120 + N, 0xF, 0xF, true));
}
template <int N>
__device__ __forceinline__ uint32_t ror(uint32_t v) {
    return static_cast<uint32_t>(
        __builtin_amdgcn_mov_dpp(static_cast<int32_t>(v), 0x120 + N, 0xF, 0xF, true));
}
__device__ __forceinline__ float lanes_max(float v) {
    v = fmaxf(v, ror<8>(v));
    v = fmaxf(v, ror<4>(v));
    v = fmaxf(v, ror<2>(v));
    return fmaxf(v, ror<1>(v));
}
__device__ __forceinline__ float lanes_sum(float v) {
    v += ror<8>(v);
    v += ror<4>(v);
    v += ror<2>(v);
    return v + ror<1>(v);
}

// exp(x) with an error of a unit and of half of |x| units; below 2^-126 it is 0.
__device__ __forceinline__ float exp_f32(float x) {
    return __builtin_amdgcn_exp2f(x * 1.44269504088896340736f);
}
__device__ __forceinline__ float sigmoid_of(float l) {
    return __builtin_amdgcn_rcpf(1.0f + exp_f32(-l));
}

template <int N>
__device__ __forceinline__ double ror(double v) {
    typedef int32_t two __attribute__((ext_vector_type(2)));
    const two w = __builtin_bit_cast(two, v);
    return __builtin_bit_cast(
        double, two{__builtin_amdgcn_mov_dpp(w[0], 0x120 + N, 0xF, 0xF, true),
                    __builtin_amdgcn_mov_dpp(w[1], 0x120 + N, 0xF, 0xF, true)});
}
// Lanes D, D + 1, ... before this one, in a circle, whose group goes before this
// lane's: a larger value, or the same and a lower index.
template <int D, class V>
__device__ __forceinline__ int lanes_ahead(V value, int j, int span) {
    if constexpr (D == kLanes) {
        return 0;
    } else {
        const V other = ror<D>(value);
        const int at = (j - D) & (kLanes - 1);
        const bool first = (other > value) | ((other == value) & (at < (j & ~(span - 1))));
        return first + lanes_ahead<D + 1, V>(value, j, span);
    }
}

__device__ __forceinline__ void order(uint32_t& a, uint32_t& b) {   // a >= b
    const uint32_t hi = max(a, b);
    b = min(a, b);
    a = hi;
}
// Descending order of N values (a power of two), by a bitonic network.
template <int N>
__device__ __forceinline__ void sort_keys(uint32_t* v) {
#pragma unroll
    for (int k = 2; k <= N; k *= 2)
#pragma unroll
        for (int j = k / 2; j > 0; j /= 2)
#pragma unroll
            for (int i = 0; i < N; ++i)
                if ((i ^ j) > i) {
                    if ((i & k) == 0)
                        order(v[i], v[i ^ j]);
                    else
                        order(v[i ^ j], v[i]);
                }
}
// The 8 largest of two descending lists, in order, into a. b is reversed
// against a, which makes the larger ones of each pair a bitonic sequence.
__device__ __forceinline__ void merge_keys(uint32_t (&a)[kList], const uint32_t (&b)[kList]) {
#pragma unroll
    for (int i = 0; i < kList; ++i) a[i] = max(a[i], b[kList - 1 - i]);
#pragma unroll
    for (int j = kList / 2; j > 0; j /= 2)
#pragma unroll
        for (int i = 0; i < kList; ++i)
            if ((i ^ j) > i) order(a[i], a[i ^ j]);
}
template <int N>
__device__ __forceinline__ void merge_lanes(uint32_t (&a)[kList]) {
    uint32_t b[kList];
#pragma unroll
    for (int i = 0; i < kList; ++i) b[i] = ror<N>(a[i]);
    merge_keys(a, b);
}

template <int VALS>
__device__ __forceinline__ void load_values(const float* p, float (&v)[VALS]) {
    struct alignas(VALS * 4 < 16 ? VALS * 4 : 16) Raw {
        float v[VALS];
    };
    const Raw r = *reinterpret_cast<const Raw*>(p);
#pragma unroll
    for (int i = 0; i < VALS; ++i) v[i] = r.v[i];
}
template <int VALS>
__device__ __forceinline__ void load_values(const __bf16* p, float (&v)[VALS]) {
    struct alignas(VALS * 2 < 16 ? VALS * 2 : 16) Raw {
        uint32_t v[VALS / 2];
    };
    const Raw r = *reinterpret_cast<const Raw*>(p);
#pragma unroll
    for (int i = 0; i < VALS; i += 2) {
        v[i] = __uint_as_float(r.v[i / 2] << 16);
        v[i + 1] = __uint_as_float(r.v[i / 2] & 0xFFFF0000u);
    }
}

template <int VALS>
__device__ __forceinline__ void store_values(float* p, const float (&v)[VALS]) {
    struct alignas(VALS * 4 < 16 ? VALS * 4 : 16) Raw {
        float v[VALS];
    };
    Raw r;
#pragma unroll
    for (int i = 0; i < VALS; ++i) r.v[i] = v[i];
    *reinterpret_cast<Raw*>(p) = r;
}
template <int VALS>
__device__ __forceinline__ void store_values(__bf16* p, const float (&v)[VALS]) {
    struct alignas(VALS * 2 < 16 ? VALS * 2 : 16) Raw {
        __bf16 v[VALS];
    };
    Raw r;
#pragma unroll
    for (int i = 0; i < VALS; ++i) r.v[i] = static_cast<__bf16>(v[i]);
    *reinterpret_cast<Raw*>(p) = r;
}

// A lane holds `per` of the experts, VALS or fewer. GROUPED needs E = 16 per and
// groups of 1, 2, 4, 8 or 16 lanes (`span`).
template <int VALS, class L, bool BY_VALUE, bool GROUPED>
__global__ __launch_bounds__(kWaves * 64)
void route_lanes_kernel(const L* __restrict__ logits, const float* __restrict__ bias, int32_t T,
                        int32_t E, int32_t K, int32_t sigmoid, int32_t renormalize, float scale,
                        int32_t groups, int32_t kept, int32_t span, int32_t per, int32_t whole,
                        int32_t* __restrict__ ids, float* __restrict__ scores) {
    const int lane = threadIdx.x & 63;
    const int j = lane & (kLanes - 1);
    const int64_t row0 =
        (int64_t(blockIdx.x) * (blockDim.x >> 6) + (threadIdx.x >> 6)) * (64 / kLanes);
    if (row0 >= T) return;
    const int64_t row = row0 + (lane >> 4);
    const bool there = row < T;
    const L* in = logits + (there ? row : T - 1) * int64_t(E);

    float l[VALS];
    const int base = j * per;           // this lane's first expert
    if (whole) {                        // E = 16 VALS, aligned
        load_values<VALS>(in + base, l);
    } else {
#pragma unroll
        for (int i = 0; i < VALS; ++i) {
            const int e = base + i;
            const float x = logit_at(in, min(e, E - 1));
            l[i] = i < per && e < E ? x : -INFINITY;
        }
    }
#pragma unroll
    for (int i = 0; i < VALS; ++i) l[i] = taking_part(l[i]);
    // The softmax's statistics over all experts.
    float top = -INFINITY, sum = 0.0f;
    if (!sigmoid) {
#pragma unroll
        for (int i = 0; i < VALS; ++i) top = fmaxf(top, l[i]);
        top = lanes_max(top);
        if (!renormalize) {
            const float from = top > -INFINITY ? top : 0.0f;
#pragma unroll
            for (int i = 0; i < VALS; ++i) sum += exp_f32(l[i] - from);
            sum = lanes_sum(sum);
        }
    }
    // v in 32 bits: the exponential and the reciprocal are off by a unit each,
    // the sums by half, |l| times half a unit enters the exponent where the
    // sigmoid's slope makes 0.23 of it: 4 half units of 1, and one of the sum with
    // the bias.
    float v[VALS];
    if constexpr (BY_VALUE) {
        float b[VALS];
        if (whole) {
            load_values<VALS>(bias + base, b);
        } else {
#pragma unroll
            for (int i = 0; i < VALS; ++i) b[i] = bias[min(base + i, E - 1)];
        }
#pragma unroll
        for (int i = 0; i < VALS; ++i) {
            const float w = sigmoid_of(l[i]) + b[i];
            v[i] = l[i] > -INFINITY && w == w ? w : -INFINITY;
        }
    } else {
#pragma unroll
        for (int i = 0; i < VALS; ++i) v[i] = l[i];
    }
    uint64_t open = ~uint64_t(0);       // lanes of the kept groups
    bool open_bad = false;
    if constexpr (GROUPED) {
        // The two largest of a group: of a lane, then of its lanes.
        float first = -INFINITY, second = -INFINITY, largest = 0.0f;
#pragma unroll
        for (int i = 0; i < VALS; ++i) {
            second = fmaxf(second, fminf(first, v[i]));
            first = fmaxf(first, v[i]);
        }
        auto join = [&](float of, float os) {
            second = fmaxf(fminf(first, of), fmaxf(second, os));
            first = fmaxf(first, of);
        };
        if (span > 1) join(__shfl_xor(first, 1, 64), __shfl_xor(second, 1, 64));
        if (span > 2) join(__shfl_xor(first, 2, 64), __shfl_xor(second, 2, 64));
        if (span > 4) join(__shfl_xor(first, 4, 64), __shfl_xor(second, 4, 64));
        if (span > 8) join(__shfl_xor(first, 8, 64), __shfl_xor(second, 8, 64));
        float value = first;
        if (sigmoid) {
            // Without a bias the two largest logits are those of the largest sigmoids.
            float a = first, b = second;
            if (!BY_VALUE) {
                if (a > -INFINITY) a = sigmoid_of(a);
                if (b > -INFINITY) b = sigmoid_of(b);
            }
            value = b > -INFINITY ? a + b : a;
            largest = lanes_max(
                fmaxf(a > -INFINITY ? fabsf(a) : 0.0f, b > -INFINITY ? fabsf(b) : 0.0f));
        }
        const float margin = sigmoid ? (8.0f + 4.0f * largest) * 0x1p-22f : 0.0f;
        bool keep = lanes_ahead<1, float>(value, j, span) < kept * span;
        if (sigmoid && kept < groups) {
            const float least = -lanes_max(keep ? -value : -INFINITY);
            const float next = lanes_max(keep ? -INFINITY : value);
            // Groups without an expert are no choice.
            open_bad = next > -INFINITY && !(least - next > margin);
            if (__any(open_bad)) {
                // The groups' values in 64 bits.
                double exact = 0.0;
                bool sure = true;
                if constexpr (BY_VALUE) {
                    // Its two largest, if no third is near the second.
                    const float from = second - margin;
                    int found = 0, one = 0, two = 0;
#pragma unroll
                    for (int i = 0; i < VALS; ++i)
                        if (v[i] > -INFINITY && v[i] >= from) {
                            two = one;
                            one = base + i;
                            ++found;
                        }
                    auto counts = [&](int e) {
                        return sigmoid_64(logit_at(in, e)) + static_cast<double>(bias[e]);
                    };
                    if (found > 0) exact = counts(one);
                    if (found > 1) exact += counts(two);
                    for (int d = 1; d < span; d *= 2) {
                        exact += __shfl_xor(exact, d, 64);
                        found += __shfl_xor(found, d, 64);
                    }
                    sure = found == (first > -INFINITY) + (second > -INFINITY);
                } else {
                    if (first > -INFINITY) exact = in_sum(first);
                    if (second > -INFINITY) exact += in_sum(second);
                }
                if (!(first > -INFINITY)) exact = -INFINITY;
                keep = lanes_ahead<1, double>(exact, j, span) < kept * span;
                open_bad = (__ballot(!sure) >> (lane & 48) & 0xFFFF) != 0;
            }
        }
        open = __ballot(keep);
#pragma unroll
        for (int i = 0; i < VALS; ++i) v[i] = keep ? v[i] : -INFINITY;
    }
    float m = v[0];
#pragma unroll
    for (int i = 1; i < VALS; ++i) m = fmaxf(m, v[i]);
    m = lanes_max(m);
    uint32_t key[VALS < kList ? kList : VALS];
#pragma unroll
    for (int i = 0; i < VALS; ++i) {
        // Below 0 and NaN become 0.
        const float d = __builtin_fmaf(v[i] - m, 0x1p20f, 16777215.0f);
        key[i] = (static_cast<uint32_t>(fmaxf(d, 0.0f)) << 8) | (255 - (base + i));
    }
    uint32_t list[kList];
    {
        uint32_t k[VALS < kList ? kList : VALS];
#pragma unroll
        for (int i = 0; i < VALS; ++i) k[i] = key[i];
#pragma unroll
        for (int i = VALS; i < kList; ++i) k[i] = 0;
        if constexpr (VALS <= kList) {
            sort_keys<VALS>(k);
#pragma unroll
            for (int i = 0; i < kList; ++i) list[i] = k[i];
        } else {
            static_assert(VALS == 2 * kList, "two lists");
            sort_keys<kList>(k);
            sort_keys<kList>(k + kList);
            uint32_t b[kList];
#pragma unroll
            for (int i = 0; i < kList; ++i) {
                list[i] = k[i];
                b[i] = k[kList + i];
            }
            merge_keys(list, b);
        }
    }
    merge_lanes<8>(list);
    merge_lanes<4>(list);
    merge_lanes<2>(list);
    merge_lanes<1>(list);
    uint32_t mine = 0, last = 0;
#pragma unroll
    for (int i = 0; i < kList; ++i) {
        if (i == j) mine = list[i];
        if (i == K - 1) last = list[i];
    }
    if (j >= K) mine = 0;
    bool bad = open_bad || last < 256;  // not K experts within 16 of the largest
    int id = j < K ? 255 - static_cast<int>(mine & 255) : -1;
    float chosen = 0.0f;
    if (j < K && id < E) chosen = taking_part(logit_at(in, id));
    // The choice against the values.
    float value = chosen;
    if constexpr (BY_VALUE) {
        value = sigmoid_of(chosen);
        if (j < K && id < E) value += bias[id];
    }
    const float next = __shfl(value, lane + 1 < 64 ? lane + 1 : lane, 64);
    const int next_id = __shfl(id, lane + 1 < 64 ? lane + 1 : lane, 64);
    const float least = __shfl(value, (lane & 48) + K - 1, 64);
    const float margin = BY_VALUE ? (4.0f + fabsf(m) + fabsf(least)) * 0x1p-22f : 0.0f;
    // The last key's value may be above another's by what a key does not hold.
    const float limit = BY_VALUE ? least - margin - 0x1p-20f : least;
    float above = -INFINITY;            // the largest of those not chosen
#pragma unroll
    for (int i = 0; i < VALS; ++i) above = fmaxf(above, key[i] < last ? v[i] : -INFINITY);
    if constexpr (BY_VALUE) {
        if (__any(above > limit || (j + 1 < K && !(value - next > margin)))) {
            // One more that may belong to the chosen goes to lane K.
            int over = 0, at = -1;
#pragma unroll
            for (int i = 0; i < VALS; ++i)
                if (key[i] < last && v[i] > limit) {
                    ++over;
                    at = base + i;
                }
            const uint32_t some = static_cast<uint32_t>(__ballot(over > 0) >> (lane & 48)) & 0xFFFF;
            const uint32_t many = static_cast<uint32_t>(__ballot(over > 1) >> (lane & 48)) & 0xFFFF;
            const bool one = __popc(some) == 1 && many == 0;
            const int more = __shfl(at, (lane & 48) + (one ? __ffs(some) - 1 : 0), 64);
            bad = bad || (some != 0 && !one);
            const int n = K + one;
            if (one && j == K) {
                id = more;
                chosen = logit_at(in, id);
            }
            // In order by the values in 64 bits; equal ones by index.
            double v64 = -INFINITY;
            if (j < n && id < E) v64 = sigmoid_64(chosen) + static_cast<double>(bias[id]);
            int before = 0;
            for (int k = 0; k <= K; ++k) {
                const double other = __shfl(v64, (lane & 48) + k, 64);
                const int other_id = __shfl(id, (lane & 48) + k, 64);
                before += other > v64 || (other == v64 && other_id < id);
            }
            const int to = (lane & 48) + (j < n ? before : j);
            id = __builtin_amdgcn_ds_permute(to * 4, id);
            chosen = __builtin_bit_cast(
                float, __builtin_amdgcn_ds_permute(to * 4, __builtin_bit_cast(int32_t, chosen)));
            if (j >= K) id = -1;
        }
    } else {
        bad = bad || above > limit ||
              (j + 1 < K && !(value > next || (value == next && id < next_id)));
    }

    // Tokens that the check does not clear, one after the other.
    const uint64_t failed = __ballot(bad && there), unsure = __ballot(open_bad);
#pragma unroll 1
    for (int r = 0; r < 64 / kLanes; ++r) {
        if (!(failed >> (r * kLanes) & 0xFFFF)) continue;
        // Groups that are certain stay as they are.
        const uint32_t certain =
            GROUPED && !(unsure >> (r * kLanes) & 1)
                ? static_cast<uint32_t>(open >> (r * kLanes)) & 0xFFFF : 0;
        const int slow = choose<(VALS + 3) / 4, L>(
            logits + (row0 + r) * E, bias, lane, K, E, sigmoid != 0, certain ? 1 : groups, kept,
            certain ? certain : 1, certain ? per : 1024);
        const int here = __shfl(slow, j, 64);
        if ((lane >> 4) == r) {
            id = j < K ? here : -1;
            chosen = id >= 0 ? logit_at(in, id) : 0.0f;
        }
    }
    float p = 0.0f;
    if (sigmoid) {
        p = chosen_sigmoid(id, chosen, renormalize, sum, lanes_max, lanes_sum);
    } else {
        if (id >= 0) p = expf(chosen - top);
        if (renormalize) sum = lanes_sum(p);
    }
    if (renormalize || !sigmoid) p = sum == 0.0f ? 0.0f : p / sum;
    if (there && j < K) {
        ids[row * K + j] = id;
        scores[row * K + j] = p * scale;
    }
}

__device__ __forceinline__ void store_grad(float* p, int64_t i, float v) { p[i] = v; }
__device__ __forceinline__ void store_grad(__bf16* p, int64_t i, float v) {
    p[i] = static_cast<__bf16>(v);
}

// With g = scale * the scores' gradient and q the scores without the scale, S
// the sum they were divided by:
//   softmax              dl_j = q_j (g_j - s) if j was chosen, else -p_j s
//   softmax, renormalized   dl_j = q_j (g_j - s), s = sum of g q, else 0
//   sigmoid              dl_j = g_j p_j (1 - p_j)
//   sigmoid, renormalized   dl_j = q_j (g_j - s) (1 - p_j)
// In the last one q_j stands for p_j / S, at most 1, since (g_j - s) / S alone
// leaves fp32 where S is small. A row is written whole; an expert in two slots gets
// the sum of both.
template <class L>
__global__ __launch_bounds__(kWaves * 64)
void route_grad_kernel(const L* __restrict__ logits, const int32_t* __restrict__ ids,
                       const float* __restrict__ grad, int32_t T, int32_t E, int32_t K,
                       int32_t sigmoid, int32_t renormalize, float scale, L* __restrict__ out) {
    const int lane = threadIdx.x & 63;
    const int64_t row = int64_t(blockIdx.x) * (blockDim.x >> 6) + (threadIdx.x >> 6);
    if (row >= T) return;
    const L* in = logits + row * E;
    const bool dense = !sigmoid && !renormalize;
    int id = -1;
    float g = 0.0f, l = -INFINITY;
    if (lane < K) {
        id = ids[row * K + lane];
        if (id < 0 || id >= E) id = -1;
        if (id >= 0) l = taking_part(logit_at(in, id));
        if (!(l > -INFINITY)) id = -1;
        if (id >= 0) g = grad[row * K + lane] * scale;
    }
    float top = -INFINITY, sum = 0.0f;
    if (dense) {
        for (int e = lane; e < E; e += 64) top = fmaxf(top, taking_part(logit_at(in, e)));
        top = wave_max(top);
        for (int e = lane; e < E; e += 64) {
            const float v = taking_part(logit_at(in, e));
            if (v > -INFINITY) sum += expf(v - top);
        }
        sum = wave_sum(sum);
    } else if (!sigmoid) {
        top = wave_max(l);
    }
    float p = 0.0f;
    if (sigmoid) {
        p = chosen_sigmoid(id, l, renormalize, sum, wave_max<float>, wave_sum);
    } else {
        if (id >= 0) p = expf(l - top);
        if (renormalize) sum = wave_sum(p);
    }
    float d = 0.0f, s = 0.0f;
    if (sigmoid) {
        const float rest = id < 0 ? 0.0f : sigmoid_rest(l);
        if (renormalize) {
            const float q = sum == 0.0f ? 0.0f : p / sum;
            s = wave_sum(g * q);
            d = sum == 0.0f ? 0.0f : (g - s) * (q * rest);
        } else {
            d = g * (p * rest);
        }
    } else {
        const float q = sum == 0.0f ? 0.0f : p / sum;
        s = wave_sum(g * q);
        d = dense ? g * q : (g - s) * q;
    }
    if (id < 0) d = 0.0f;
    for (int base = 0; base < E; base += 64) {
        const int e = base + lane;
        float v = 0.0f;
        if (dense && e < E) {
            const float x = taking_part(logit_at(in, e));
            if (x > -INFINITY) v = -(expf(x - top) / sum) * s;
        }
        for (int k = 0; k < K; ++k) {
            const float dk = __shfl(d, k, 64);
            if (__shfl(id, k, 64) == e) v += dk;
        }
        if (e < E) store_grad(out, row * E + e, v);
    }
}

// The same for up to 256 experts, 16 lanes per token as in the choice; lane j also
// holds slot j. Bound: the launch; 8191 tokens of 128 experts, 8 each, bf16, softmax
// renormalized 4.4 us on MI355X.
template <int VALS, class L>
__global__ __launch_bounds__(kWaves * 64)
void route_grad_lanes_kernel(const L* __restrict__ logits, const int32_t* __restrict__ ids,
                             const float* __restrict__ grad, int32_t T, int32_t E, int32_t K,
                             int32_t sigmoid, int32_t renormalize, float scale, int32_t whole,
                             L* __restrict__ out) {
    const int lane = threadIdx.x & 63;
    const int j = lane & (kLanes - 1);
    const int64_t row0 =
        (int64_t(blockIdx.x) * (blockDim.x >> 6) + (threadIdx.x >> 6)) * (64 / kLanes);
    if (row0 >= T) return;
    const bool there = row0 + (lane >> 4) < T;
    const int64_t row = there ? row0 + (lane >> 4) : T - 1;
    const L* in = logits + row * E;
    const bool dense = !sigmoid && !renormalize;
    int id = -1;
    float g = 0.0f, l = -INFINITY;
    if (j < K) {
        id = ids[row * K + j];
        g = grad[row * K + j] * scale;
        if (id < 0 || id >= E) id = -1;
        if (id >= 0) l = taking_part(logit_at(in, id));
        if (!(l > -INFINITY)) id = -1;
        if (id < 0) g = 0.0f;
    }
    float v[VALS];
    float top = -INFINITY, sum = 0.0f;
    if (dense) {
        if (whole) {
            load_values<VALS>(in + j * VALS, v);
        } else {
#pragma unroll
            for (int i = 0; i < VALS; ++i) {
                const int e = j * VALS + i;
                const float x = logit_at(in, min(e, E - 1));
                v[i] = e < E ? x : -INFINITY;
            }
        }
#pragma unroll
        for (int i = 0; i < VALS; ++i) top = fmaxf(top, v[i] = taking_part(v[i]));
        top = lanes_max(top);
        const float from = top > -INFINITY ? top : 0.0f;
#pragma unroll
        for (int i = 0; i < VALS; ++i) sum += v[i] = exp_f32(v[i] - from);
        sum = lanes_sum(sum);
    } else if (!sigmoid) {
        top = lanes_max(l);
    }
    float p = 0.0f;
    if (sigmoid) {
        p = chosen_sigmoid(id, l, renormalize, sum, lanes_max, lanes_sum);
    } else {
        if (id >= 0) p = expf(l - top);
        if (renormalize) sum = lanes_sum(p);
    }
    float d, s = 0.0f;
    if (sigmoid) {
        const float rest = id < 0 ? 0.0f : sigmoid_rest(l);
        if (renormalize) {
            const float q = sum == 0.0f ? 0.0f : p / sum;
            s = lanes_sum(g * q);
            d = sum == 0.0f ? 0.0f : (g - s) * (q * rest);
        } else {
            d = g * (p * rest);
        }
    } else {
        const float q = sum == 0.0f ? 0.0f : p / sum;
        s = lanes_sum(g * q);
        d = dense ? g * q : (g - s) * q;
    }
    if (id < 0) d = 0.0f;
    const float share = dense && sum > 0.0f ? -s / sum : 0.0f;
#pragma unroll
    for (int i = 0; i < VALS; ++i) v[i] = dense ? v[i] * share : 0.0f;
    const int first = j * VALS;
    for (int k = 0; k < K; ++k) {
        const float dk = __shfl(d, (lane & 48) + k, 64);
        const int at = __shfl(id, (lane & 48) + k, 64) - first;
#pragma unroll
        for (int i = 0; i < VALS; ++i)
            if (at == i) v[i] += dk;
    }
    if (!there) return;
    if (whole) {
        store_values<VALS>(out + row * E + first, v);
    } else {
#pragma unroll
        for (int i = 0; i < VALS; ++i)
            if (first + i < E) store_grad(out, row * E + first + i, v[i]);
    }
}

// A wavefront per workgroup until there is one for every SIMD.
int lane_waves(int32_t T) { return T <= 4 * 1024 ? 1 : kWaves; }
int lane_values(int32_t E) {
    return E <= kLanes * 2 ? 2 : E <= kLanes * 4 ? 4 : E <= kLanes * 8 ? 8 : 16;
}

template <int VALS, class L>
hipError_t launch_lanes(const RouteArgs& a, int32_t per, hipStream_t stream) {
    const bool by_value = a.sigmoid && a.bias, grouped = a.groups > 1;
    auto kernel = by_value ? (grouped ? route_lanes_kernel<VALS, L, true, true>
                                      : route_lanes_kernel<VALS, L, true, false>)
                           : (grouped ? route_lanes_kernel<VALS, L, false, true>
                                      : route_lanes_kernel<VALS, L, false, false>);
    const bool whole = a.E == kLanes * VALS && reinterpret_cast<uintptr_t>(a.logits) % 16 == 0 &&
                       reinterpret_cast<uintptr_t>(a.bias) % 16 == 0;
    const int waves = lane_waves(a.T);
    const int64_t tokens = waves * (64 / kLanes);
    hipLaunchKernelGGL(kernel, dim3(static_cast<uint32_t>((a.T + tokens - 1) / tokens)),
                       dim3(waves * 64), 0, stream, static_cast<const L*>(a.logits), a.bias, a.T,
                       a.E, a.K, a.sigmoid, a.renormalize, a.scale, a.groups, a.kept,
                       kLanes / a.groups, per, whole, a.ids, a.scores);
    return hipGetLastError();
}

// Experts of a lane if the 16 lanes of a token can take its groups, else 0.
int32_t lane_experts(const RouteArgs& a, int vals) {
    if (a.groups == 1) return vals;
    return a.E % kLanes == 0 && kLanes % a.groups == 0 ? a.E / kLanes : 0;
}

// Wavefronts per workgroup with one token each: one where whole workgroups of kWaves
// would make a launch of 2^32 threads.
uint32_t token_waves(int32_t T) { return (int64_t(T) + kWaves - 1) * 64 > kMaxGrid ? 1 : kWaves; }

template <int VALS, class L>
hipError_t launch_route(const RouteArgs& a, hipStream_t stream) {
    const uint32_t waves = token_waves(a.T);
    hipLaunchKernelGGL((route_kernel<VALS, L>),
                       dim3((static_cast<uint32_t>(a.T) + waves - 1) / waves), dim3(waves * 64), 0,
                       stream, static_cast<const L*>(a.logits), a.bias, a.T, a.E, a.K, a.sigmoid,
                       a.renormalize, a.scale, a.groups, a.kept, a.ids, a.scores);
    return hipGetLastError();
}

template <class L>
hipError_t route(const RouteArgs& a, hipStream_t stream) {
    if (a.E <= kLanes * 16 && a.K <= kList) {
        const int vals = lane_values(a.E);
        if (const int32_t per = lane_experts(a, vals)) {
            if (vals == 2) return launch_lanes<2, L>(a, per, stream);
            if (vals == 4) return launch_lanes<4, L>(a, per, stream);
            if (vals == 8) return launch_lanes<8, L>(a, per, stream);
            return launch_lanes<16, L>(a, per, stream);
        }
    }
    if (a.E <= 64) return launch_route<1, L>(a, stream);
    if (a.E <= 128) return launch_route<2, L>(a, stream);
    if (a.E <= 256) return launch_route<4, L>(a, stream);
    if (a.E <= 512) return launch_route<8, L>(a, stream);
    return launch_route<16, L>(a, stream);
}

template <class L>
hipError_t route_grad(const RouteGradArgs& a, hipStream_t stream) {
    if (a.E <= kLanes * 16) {
        const int vals = lane_values(a.E), waves = lane_waves(a.T);
        auto kernel = vals == 2   ? route_grad_lanes_kernel<2, L>
                      : vals == 4 ? route_grad_lanes_kernel<4, L>
                      : vals == 8 ? route_grad_lanes_kernel<8, L>
                                  : route_grad_lanes_kernel<16, L>;
        const bool whole = a.E == kLanes * vals &&
                           reinterpret_cast<uintptr_t>(a.logits) % 16 == 0 &&
                           reinterpret_cast<uintptr_t>(a.grad_logits) % 16 == 0;
        const int64_t tokens = waves * (64 / kLanes);
        hipLaunchKernelGGL(kernel, dim3(static_cast<uint32_t>((a.T + tokens - 1) / tokens)),
                           dim3(waves * 64), 0, stream, static_cast<const L*>(a.logits), a.ids,
                           a.grad, a.T, a.E, a.K, a.sigmoid, a.renormalize, a.scale, whole,
                           static_cast<L*>(a.grad_logits));
        return hipGetLastError();
    }
    const uint32_t waves = token_waves(a.T);
    hipLaunchKernelGGL((route_grad_kernel<L>),
                       dim3((static_cast<uint32_t>(a.T) + waves - 1) / waves), dim3(waves * 64), 0,
                       stream, static_cast<const L*>(a.logits), a.ids, a.grad, a.T, a.E, a.K,
                       a.sigmoid, a.renormalize, a.scale, static_cast<L*>(a.grad_logits));
    return hipGetLastError();
}

}  // namespace

hipError_t launch_route_topk(const RouteArgs& a, hipStream_t stream) {
    return a.bf16 ? route<__bf16>(a, stream) : route<float>(a, stream);
}

hipError_t launch_route_topk_grad(const RouteGradArgs& a, hipStream_t stream) {
    return a.bf16 ? route_grad<__bf16>(a, stream) : route_grad<float>(a, stream);
}

}  // namespace moe
