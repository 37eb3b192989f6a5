// The router on gfx950: the K experts of every token and their scores from the
// router's logits, and the gradient of the logits.
//
// With l the logits of a token, the experts taking part being those whose l is
// neither NaN nor -inf:
//   softmax   p = exp(l - m) / sum of exp(l - m), m the largest l
//   sigmoid   p = 1 / (1 + exp(-l))
// The K largest of v are chosen, equal ones by index; v is l where p only has
// to keep its order, else sigmoid(l) + bias. That is computed in 64 bits, so
// that the order of near values is that of the formula and not that of an
// exponential's last digit. With groups of consecutive experts only those of
// the `kept` best groups can be chosen, by the group's largest v (softmax) or the
// sum of its two largest (sigmoid).
//
// One wavefront per token; lane j holds experts j, j + 64, ...
#include <cmath>

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

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor(v, d, 64));
    return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d, 64);
    return v;
}

// The largest of the lanes' values and, of equal ones, the lowest index.
template <class V>
__device__ __forceinline__ void wave_best(V& v, int& at) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) {
        const V ov = __shfl_xor(v, d, 64);
        const int oi = __shfl_xor(at, d, 64);
        if (ov > v || (ov == v && oi < at)) {
            v = ov;
            at = oi;
        }
    }
}

// The wavefront's best of v and its expert; at least one of the lanes' own
// experts is named even where all hold -inf.
template <int VALS, class V>
__device__ __forceinline__ void best_of(const V (&v)[VALS], int lane, V& top, int& at) {
    top = v[0];
    at = lane;
#pragma unroll
    for (int i = 1; i < VALS; ++i)
        if (v[i] > top) {
            top = v[i];
            at = i * 64 + lane;
        }
    wave_best(top, at);
}

template <int VALS, class V>
__device__ __forceinline__ void take_out(V (&v)[VALS], int lane, int at) {
#pragma unroll
    for (int i = 0; i < VALS; ++i)
        if (i * 64 + lane == at) v[i] = -INFINITY;
}

// The experts chosen by v (destroyed): lane k gets the k-th, or -1.
template <int VALS, class V>
__device__ int select(V (&v)[VALS], int lane, int K, int E, int groups, int kept, bool pairs) {
    if (groups > 1) {
        const int size = E / groups;
        // Lane g holds group g's value; groups without an expert keep -inf.
        V value = -INFINITY;
        for (int g = 0; g < groups; ++g) {
            V w[VALS];
#pragma unroll
            for (int i = 0; i < VALS; ++i) {
                const int e = i * 64 + lane;
                w[i] = e >= g * size && e < (g + 1) * size ? v[i] : V(-INFINITY);
            }
            V first, second = -INFINITY;
            int at, unused;
            best_of<VALS, V>(w, lane, first, at);
            if (pairs && size > 1) {
                take_out<VALS, V>(w, lane, at);
                best_of<VALS, V>(w, lane, second, unused);
                if (second > V(-INFINITY)) first += second;
            }
            if (lane == g) value = first;
        }
        uint64_t open = 0;
        for (int j = 0; j < kept; ++j) {
            V top = value;
            int at = lane;
            wave_best(top, at);
            if (!(top > V(-INFINITY))) break;
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
        best_of<VALS, V>(v, lane, top, at);
        if (!(top > V(-INFINITY))) break;
        if (lane == k) mine = at;
        take_out<VALS, V>(v, lane, at);
    }
    return mine;
}

// The score of a chosen expert in lanes 0 .. K - 1 (id >= 0, logit l), before
// the scale; `top` and `sum` are the softmax's over all experts.
__device__ __forceinline__ float score_of(bool sigmoid, bool renormalize, int id, float l,
                                          float top, float sum) {
    float p = 0.0f;
    if (id >= 0) p = sigmoid ? 1.0f / (1.0f + expf(-l)) : expf(l - top);
    if (renormalize) sum = wave_sum(p);
    if (renormalize || !sigmoid) p = sum == 0.0f ? 0.0f : p / sum;
    return p;
}

template <int VALS, class L>
__global__ __launch_bounds__(kWaves * 64)
void route_kernel(const L* __restrict__ logits, const float* __restrict__ bias, int32_t T,
                  int32_t E, int32_t K, int32_t sigmoid, int32_t renormalize, float scale,
                  int32_t groups, int32_t kept, int32_t* __restrict__ ids,
                  float* __restrict__ scores) {
    const int lane = threadIdx.x & 63;
    const int64_t row = int64_t(blockIdx.x) * kWaves + (threadIdx.x >> 6);
    if (row >= T) return;
    const L* in = logits + row * E;
    float l[VALS];
#pragma unroll
    for (int i = 0; i < VALS; ++i) {
        const int e = i * 64 + lane;
        l[i] = e < E ? taking_part(logit_at(in, e)) : -INFINITY;
    }
    float top = 0.0f, sum = 0.0f;
    if (!sigmoid) {
        top = l[0];
#pragma unroll
        for (int i = 1; i < VALS; ++i) top = fmaxf(top, l[i]);
        top = wave_max(top);
        if (!renormalize && top > -INFINITY) {
#pragma unroll
            for (int i = 0; i < VALS; ++i)
                if (l[i] > -INFINITY) sum += expf(l[i] - top);
            sum = wave_sum(sum);
        }
    }
    int id;
    if (sigmoid && (bias || groups > 1)) {
        double v[VALS];
#pragma unroll
        for (int i = 0; i < VALS; ++i) {
            const int e = i * 64 + lane;
            v[i] = -INFINITY;
            if (l[i] > -INFINITY) {
                v[i] = 1.0 / (1.0 + exp(-static_cast<double>(l[i])));
                if (bias) v[i] += static_cast<double>(bias[e]);
                if (!(v[i] == v[i])) v[i] = -INFINITY;
            }
        }
        id = select<VALS, double>(v, lane, K, E, groups, kept, true);
    } else {
        id = select<VALS, float>(l, lane, K, E, groups, kept, sigmoid != 0);
    }
    float p = 0.0f;
    if (id >= 0) p = logit_at(in, id);
    p = score_of(sigmoid, renormalize, id, p, top, sum);
    if (lane < K) {
        ids[row * K + lane] = id;
        scores[row * K + lane] = p * scale;
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
//   sigmoid, renormalized   dl_j = (g_j - s) / S p_j (1 - p_j)
// A row is written whole; an expert in two slots gets the sum of both.
template <class L>
__global__ __launch_bounds__(kWaves * 64)
void route_grad_kernel(const L* __restrict__ logits, const int32_t* __restrict__ ids,
                       const float* __restrict__ grad, int32_t T, int32_t E, int32_t K,
                       int32_t sigmoid, int32_t renormalize, float scale, L* __restrict__ out) {
    const int lane = threadIdx.x & 63;
    const int64_t row = int64_t(blockIdx.x) * kWaves + (threadIdx.x >> 6);
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
    const float p = id < 0 ? 0.0f : sigmoid ? 1.0f / (1.0f + expf(-l)) : expf(l - top);
    if (renormalize) sum = wave_sum(p);
    float d = 0.0f, s = 0.0f;
    if (sigmoid) {
        // p (1 - p) without the difference, which loses p's last digits near 1.
        const float slope = id < 0 ? 0.0f : p / (1.0f + expf(l));
        if (renormalize) {
            s = wave_sum(sum == 0.0f ? 0.0f : g * (p / sum));
            d = sum == 0.0f ? 0.0f : (g - s) / sum * slope;
        } else {
            d = g * slope;
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

template <int VALS, class L>
hipError_t launch_route(const RouteArgs& a, hipStream_t stream) {
    hipLaunchKernelGGL((route_kernel<VALS, L>), dim3((static_cast<uint32_t>(a.T) + kWaves - 1) / kWaves),
                       dim3(kWaves * 64), 0, stream, static_cast<const L*>(a.logits), a.bias, a.T,
                       a.E, a.K, a.sigmoid, a.renormalize, a.scale, a.groups, a.kept, a.ids,
                       a.scores);
    return hipGetLastError();
}

template <class L>
hipError_t route(const RouteArgs& a, hipStream_t stream) {
    if (a.E <= 64) return launch_route<1, L>(a, stream);
    if (a.E <= 128) return launch_route<2, L>(a, stream);
    if (a.E <= 256) return launch_route<4, L>(a, stream);
    if (a.E <= 512) return launch_route<8, L>(a, stream);
    return launch_route<16, L>(a, stream);
}

template <class L>
hipError_t route_grad(const RouteGradArgs& a, hipStream_t stream) {
    hipLaunchKernelGGL((route_grad_kernel<L>), dim3((static_cast<uint32_t>(a.T) + kWaves - 1) / kWaves),
                       dim3(kWaves * 64), 0, stream, static_cast<const L*>(a.logits), a.ids, a.grad,
                       a.T, a.E, a.K, a.sigmoid, a.renormalize, a.scale,
                       static_cast<L*>(a.grad_logits));
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
