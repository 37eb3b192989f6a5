// Device building blocks of the expert feed-forward kernels on gfx950: the
// tile a workgroup owns, operand tiles in LDS filled by direct global-to-LDS
// loads, and the activation. Internal to libmoe_layout.so.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "moe_lanes.h"

namespace moe {

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int32_t v2i __attribute__((ext_vector_type(2)));

constexpr int kExpertXcds = 8;  // MI355X: 8 XCDs, each with its own L2

// Rows [s0, s1) of expert e, clamped into [0, max_rows).
__device__ __forceinline__ void expert_segment(const int32_t* offsets, int32_t e,
                                               int32_t max_rows, int32_t& s0, int32_t& s1) {
    const int32_t a = offsets[e], b = offsets[e + 1];
    s0 = min(max(a, 0), max_rows);
    s1 = min(max(b, s0), max_rows);
}

// The tile of a workgroup: expert, feature tile, first row and rows; e < 0
// marks one of the `spare` workgroups without a tile (number `f` of them) and
// row0 is then the first row of no expert.
struct ExpertTile {
    int32_t e, f, row0, rows;
};

// Finds tile number u of the launch (wavefront 0 calls it; every lane gets the
// result). Expert e owns ceil(rows / bt) * ftiles consecutive numbers; inside
// an expert, blocks of up to `band` row tiles: all feature tiles of a band,
// each with the band's row tiles fastest.
__device__ inline ExpertTile expert_find_tile(const int32_t* offsets, int32_t E, int32_t max_rows,
                                              int32_t bt, int32_t ftiles, int32_t band, int64_t u) {
    const int lane = threadIdx.x & 63;
    const int per = (E + 63) / 64;
    const int e_lo = min(E, lane * per);
    const int e_hi = min(E, e_lo + per);
    int64_t local = 0;
    for (int e = e_lo; e < e_hi; ++e) {
        int32_t s0, s1;
        expert_segment(offsets, e, max_rows, s0, s1);
        local += int64_t((s1 - s0 + bt - 1) / bt) * ftiles;
    }
    int64_t incl = local;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int64_t v = __shfl_up(incl, d, 64);
        if (lane >= d) incl += v;
    }
    const int64_t total = __shfl(incl, 63, 64);
    ExpertTile t = {-1, 0, 0, 0};
    if (u >= total) {
        t.f = static_cast<int32_t>(u - total);
        t.rows = static_cast<int32_t>(total);
        const int32_t end = offsets[E];
        t.row0 = min(max(end, 0), max_rows);
        return t;
    }
    int64_t base = incl - local;
    const bool mine = u >= base && u < incl;
    if (mine) {
        for (int e = e_lo; e < e_hi; ++e) {
            int32_t s0, s1;
            expert_segment(offsets, e, max_rows, s0, s1);
            const int32_t mt = (s1 - s0 + bt - 1) / bt;
            const int64_t n = int64_t(mt) * ftiles;
            if (u < base + n) {
                const int64_t rem = u - base;
                const int32_t mb = static_cast<int32_t>(rem / (int64_t(ftiles) * band));
                const int32_t in = static_cast<int32_t>(rem - int64_t(mb) * ftiles * band);
                const int32_t mbe = min(band, mt - mb * band);
                t.e = e;
                t.f = in / mbe;
                t.row0 = s0 + (mb * band + in % mbe) * bt;
                t.rows = min(bt, s1 - t.row0);
                break;
            }
            base += n;
        }
    }
    const int src = __ffsll(static_cast<unsigned long long>(__ballot(mine))) - 1;
    t.e = __shfl(t.e, src, 64);
    t.f = __shfl(t.f, src, 64);
    t.row0 = __shfl(t.row0, src, 64);
    t.rows = __shfl(t.rows, src, 64);
    return t;
}

// Workgroup b runs on XCD b % 8; XCD x takes chunks x, x + 8, ... of `chunk`
// tile numbers (the grid holds whole chunks per XCD), so the tiles one XCD
// runs at once are neighbours and share its L2.
__device__ __forceinline__ int64_t expert_tile_number(int32_t chunk) {
    const int64_t idx = blockIdx.x / kExpertXcds;
    const int64_t x = blockIdx.x % kExpertXcds;
    return ((idx / chunk) * kExpertXcds + x) * chunk + idx % chunk;
}

// +0.0 into rows [row0, max_rows) of `width` 16-byte chunks, spread over the
// workgroups without a tile (this one is number `index` of `count`).
__device__ __forceinline__ void expert_zero_tail(v4i* out, int64_t row0, int64_t max_rows,
                                                 int32_t width, int64_t index, int64_t count) {
    const v4i zero = {0, 0, 0, 0};
    for (int64_t r = row0 + index; r < max_rows; r += count)
        for (int32_t c = threadIdx.x; c < width; c += blockDim.x) out[r * width + c] = zero;
}

typedef __attribute__((address_space(3))) v4i lds_v4i;
typedef __attribute__((address_space(3))) bf16x4 lds_bf16x4;

// Asynchronous 16-byte load of every lane into LDS: lane l's bytes land at
// dst + 16 l (dst is the same for the whole wavefront).
__device__ __forceinline__ void load_to_lds(const char* src, v4i* dst) {
    __builtin_amdgcn_global_load_lds(
        (const __attribute__((address_space(1))) void*)(src),
        (__attribute__((address_space(3))) void*)(dst), 16, 0, 0);
}

// Barrier without the full memory drain of __syncthreads(): loads in flight
// into other buffers stay in flight. The empty asm statements keep the
// compiler from moving LDS accesses across it.
__device__ __forceinline__ void step_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Waits until at most N of this wavefront's global loads are in flight and
// all its LDS reads have returned.
template <int N>
__device__ __forceinline__ void wait_loads() {
    // vmcnt in bits 3:0 and 15:14, expcnt (6:4) left open, lgkmcnt (11:8) 0.
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
}

// Waits until all this wavefront's LDS reads have returned.
__device__ __forceinline__ void wait_lds_reads() {
    __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4));
}

// An operand whose sum index is contiguous in memory: EXT positions (rows or
// features) x 64 elements of the sum, 128 bytes per position. 16-byte chunk c
// of position p sits at chunk c ^ swz(p), which makes the fragment reads (16
// consecutive positions at one chunk) hit 16 distinct bank groups. A direct
// load writes 64 consecutive chunks, so the swizzle is applied to the address
// each lane reads.
template <int EXT, int WAVES>
struct PackedOperand {
    static constexpr int kChunks = EXT * 8;
    static constexpr int kLoads = EXT / (8 * WAVES);
    static_assert(EXT % (8 * WAVES) == 0, "whole wavefront loads");
    const char* base[kLoads];  // wavefront-uniform
    uint32_t off[kLoads];
    int32_t chunk[kLoads];
    int wave;
    uint32_t frag_at[2];       // chunk of this lane's fragment, halves of a step

    __device__ static int swz(int p) { return ((p & 15) ^ ((p & 15) >> 3)) & 7; }

    // row(p) gives the matrix row of position p relative to base_of(p); both
    // are uniform over groups of 8 positions except for the row itself.
    template <class Base, class Row>
    __device__ void init(int wave_, int lane, int64_t pitch, Base base_of, Row row) {
        wave = wave_;
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int p0 = (wave + WAVES * j) * 8;
            const int p = p0 + (lane >> 3);
            chunk[j] = (lane & 7) ^ swz(p);
            base[j] = base_of(p0);
            off[j] = static_cast<uint32_t>(row(p) * pitch) + chunk[j] * 16;
        }
        const int i = lane & 15, g = lane >> 4;
#pragma unroll
        for (int s = 0; s < 2; ++s) frag_at[s] = i * 8 + ((4 * s + g) ^ swz(i));
    }
    __device__ void issue(int64_t step, v4i* buf) const {
#pragma unroll
        for (int j = 0; j < kLoads; ++j)
            load_to_lds(base[j] + step * 128 + off[j], buf + (wave + WAVES * j) * 64);
    }
    // The last, partial step: chunks at or past `chunks` of the row are zero.
    __device__ void tail(int64_t step, int32_t chunks, int lane, v4i* buf) const {
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            v4i v = {0, 0, 0, 0};
            if (step * 8 + chunk[j] < chunks)
                v = *reinterpret_cast<const v4i*>(base[j] + step * 128 + off[j]);
            buf[(wave + WAVES * j) * 64 + lane] = v;
        }
    }
    // Positions [16 blk, 16 blk + 16), half s of the step.
    __device__ bf16x8 frag(const v4i* buf, int blk, int s) const {
        return __builtin_bit_cast(bf16x8, buf[frag_at[s] + blk * 128]);
    }
};

// An operand whose sum index strides in memory: 64 rows of the sum x EXT
// contiguous positions. Fragments come out of LDS transposed (ds_read_b64_tr:
// a group of 16 lanes reads 4 sum rows of 32 bytes and each lane receives one
// position's 4 elements). The 32-byte blocks of a sum row are stored at block
// b ^ f(row) with f(row) = row % 4 + 4 * (row / 8 % 2): the 8 sum rows two
// lane groups read together then lie in distinct banks.
template <int EXT, int WAVES>
struct StridedOperand {
    static constexpr int kRowChunks = EXT / 8;
    static constexpr int kChunks = 64 * kRowChunks;
    static constexpr int kLoads = kChunks / (64 * WAVES);
    static_assert(EXT % 128 == 0 && kChunks % (64 * WAVES) == 0, "whole wavefront loads");
    const char* base;          // wavefront-uniform
    int64_t step_bytes;
    uint32_t off[kLoads];
    int wave;
    uint32_t frag_row;         // byte of this lane's first sum row
    int fx;                    // this lane's block swizzle

    __device__ static int fswz(int k) { return (k & 3) | ((k >> 1) & 4); }

    // base_: element (first sum row, first position) of the tile; positions
    // at or past `width` (a multiple of 8) read the last valid chunk.
    __device__ void init(int wave_, int lane, int64_t pitch, const char* base_, int32_t width) {
        wave = wave_;
        base = base_;
        step_bytes = pitch * 64;
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int q = (wave + WAVES * j) * 64 + lane;
            const int k = q / kRowChunks, pos = q % kRowChunks;
            const int c = (((pos >> 1) ^ fswz(k)) << 1) | (pos & 1);
            off[j] = static_cast<uint32_t>(k * pitch) + min(c, width / 8 - 1) * 16;
        }
        const int i = lane & 15, g = lane >> 4;
        fx = (i >> 2) | ((g & 1) << 2);
        frag_row = (8 * g + (i >> 2)) * (EXT * 2) + (i & 3) * 8;
    }
    __device__ void issue(int64_t step, v4i* buf) const {
#pragma unroll
        for (int j = 0; j < kLoads; ++j)
            load_to_lds(base + step * step_bytes + off[j], buf + (wave + WAVES * j) * 64);
    }
    // The last, partial step: sum rows at or past `rows` (counted from the
    // first step) are zero.
    __device__ void tail(int64_t step, int64_t rows, int lane, v4i* buf) const {
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int q = (wave + WAVES * j) * 64 + lane;
            v4i v = {0, 0, 0, 0};
            if (step * 64 + q / kRowChunks < rows)
                v = *reinterpret_cast<const v4i*>(base + step * step_bytes + off[j]);
            buf[q] = v;
        }
    }
    __device__ bf16x8 frag(const v4i* buf, int blk, int s) const {
        const char* p = reinterpret_cast<const char*>(buf) + frag_row + ((blk ^ fx) * 32) +
                        s * (32 * EXT * 2);
        const bf16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)(p));
        const bf16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)(p + 4 * EXT * 2));
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
};

// act(g) and its derivative in fp32. silu(g) = g sigmoid(g); the tanh form of
// gelu is g sigmoid(2z) with z = sqrt(2/pi) (g + 0.044715 g^3), which loses no
// digits where 1 + tanh(z) would cancel. exp runs to infinity or zero at the
// ends, where the sigmoid is exactly 0 or 1.
constexpr int kActSilu = 0;
constexpr int kActGelu = 1;
__device__ __forceinline__ float sigmoid_f32(float z) {
    return __builtin_amdgcn_rcpf(1.0f + __expf(-z));
}
__device__ __forceinline__ float activate(int act, float g) {
    float z = g;
    if (act == kActGelu) z = 1.5957691216057308f * __builtin_fmaf(0.044715f * g * g, g, g);
    return g * sigmoid_f32(z);
}
__device__ __forceinline__ void activate_grad(int act, float g, float& value, float& slope) {
    float z = g, dz = 1.0f;
    if (act == kActGelu) {
        const float g2 = g * g;
        z = 1.5957691216057308f * __builtin_fmaf(0.044715f * g2, g, g);
        dz = 1.5957691216057308f * __builtin_fmaf(3.0f * 0.044715f, g2, 1.0f);
    }
    const float p = sigmoid_f32(z);
    const float pq = p * (1.0f - p);
    value = g * p;
    // Where the sigmoid has saturated its slope is 0 whatever dz overflows to.
    slope = pq == 0.0f ? p : __builtin_fmaf(g * pq, dz, p);
}

__device__ __forceinline__ v2i pack_bf16x4(float a, float b, float c, float d) {
    v2i v;
    v[0] = static_cast<int32_t>(f32_to_bf16_bits(a) | (f32_to_bf16_bits(b) << 16));
    v[1] = static_cast<int32_t>(f32_to_bf16_bits(c) | (f32_to_bf16_bits(d) << 16));
    return v;
}

}  // namespace moe
