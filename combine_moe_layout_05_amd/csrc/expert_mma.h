// Device building blocks of the expert feed-forward kernels on gfx950: the
// tile a workgroup owns, operand tiles in LDS filled by direct global-to-LDS
// loads, and the activation. Internal to libmoe_layout.so.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "expert_kernels.h"
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
// each with the band's row tiles fastest. A lane holds up to 16 neighbouring
// experts; their offsets are loaded in groups of 4, together, since every
// workgroup waits for this before its first useful load.
__device__ inline ExpertTile expert_find_tile(const int32_t* offsets, int32_t E, int32_t max_rows,
                                              int32_t bt, int32_t ftiles, int32_t band, int64_t u) {
    constexpr int kGroup = 4;
    const int lane = threadIdx.x & 63;
    const int per = (E + 63) / 64;
    const int e_lo = min(E, lane * per);
    const int e_hi = min(E, e_lo + per);
    int32_t first[kGroup + 1];              // first row of the group's experts
    auto load_group = [&](int e0) {
#pragma unroll
        for (int k = 0; k <= kGroup; ++k) first[k] = offsets[min(e0 + k, E)];
#pragma unroll
        for (int k = 0; k <= kGroup; ++k) first[k] = min(max(first[k], 0), max_rows);
    };
    auto tiles_of = [&](int e0, int k) -> int32_t {
        return e0 + k < e_hi ? expert_row_parts(max(first[k + 1] - first[k], 0), bt) : 0;
    };
    const int32_t end = min(max(offsets[E], 0), max_rows);
    int64_t local = 0;
    for (int e0 = e_lo; e0 < max(e_hi, e_lo + 1); e0 += kGroup) {
        load_group(e0);
#pragma unroll
        for (int k = 0; k < kGroup; ++k) local += int64_t(tiles_of(e0, k)) * ftiles;
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
        t.row0 = end;
        return t;
    }
    int64_t base = incl - local;
    const bool mine = u >= base && u < incl;
    if (mine) {
        for (int e0 = e_lo; e0 < e_hi; e0 += kGroup) {
            if (per > kGroup) load_group(e0);
#pragma unroll
            for (int k = 0; k < kGroup; ++k) {
                const int32_t mt = tiles_of(e0, k);
                const int64_t rem = u - base;
                base += int64_t(mt) * ftiles;
                if (rem >= 0 && rem < int64_t(mt) * ftiles) {
                    const int32_t mb = static_cast<int32_t>(rem / (int64_t(ftiles) * band));
                    const int32_t in = static_cast<int32_t>(rem - int64_t(mb) * ftiles * band);
                    const int32_t mbe = min(band, mt - mb * band);
                    t.e = e0 + k;
                    t.f = in / mbe;
                    t.row0 = first[k] + (mb * band + in % mbe) * bt;
                    t.rows = min(bt, first[k + 1] - t.row0);
                }
            }
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

// +0.0 into rows of no segment, of `width` 16-byte chunks each: from `end` on
// (kZeroTail in `zero`), before the first segment (kZeroHead). Spread over the
// workgroups without a tile (this one is number `index` of `count`).
__device__ __forceinline__ void expert_zero_rows(v4i* out, const int32_t* offsets, int32_t zero,
                                                 int64_t end, int64_t max_rows, int32_t width,
                                                 int64_t index, int64_t count) {
    const v4i nothing = {0, 0, 0, 0};
    auto clear = [&](int64_t from, int64_t to) {
        for (int64_t r = from + index; r < to; r += count)
            for (int32_t c = threadIdx.x; c < width; c += blockDim.x) out[r * width + c] = nothing;
    };
    if (zero & kZeroTail) clear(end, max_rows);
    if (zero & kZeroHead) clear(0, min(static_cast<int64_t>(offsets[0]), end));
}

typedef __attribute__((address_space(3))) v4i lds_v4i;
typedef __attribute__((address_space(3))) bf16x4 lds_bf16x4;

// Asynchronous 16-byte load of every lane into LDS: lane l reads base + off and
// its bytes land at dst + 16 l (base and dst are the same for the whole
// wavefront). The instruction has no register result; its bytes are in LDS once
// wait_loads() has seen it finish (and, for other wavefronts, after a barrier
// behind that). Written out, since the compiler's own form of it makes every
// later LDS read wait for all such loads wherever control flow joins, which
// takes the loads of later steps out of flight.
//
// A memory instruction may read a scalar register no sooner than 5 wait states
// after a vector instruction wrote it (here v_readfirstlane, with which the
// compiler may form the base right in front); nothing but the code keeps that
// distance, and the compiler does not look inside the statement. s_nop 4 is 5
// wait states, one of which the write of m0 needs as well.
__device__ __forceinline__ void load_to_lds(const char* base, uint32_t off, v4i* dst) {
    const uint32_t lds = static_cast<uint32_t>(
        reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) void*)(dst)));
    const uint64_t b = reinterpret_cast<uint64_t>(base);
    const uint64_t lo =
        static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(b)));
    const uint64_t hi =
        static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(b >> 32)));
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, %2"
                 :
                 : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(off), "s"(lo | (hi << 32))
                 : "memory", "m0");
}

// The value of a register, as something the compiler knows nothing about: what
// is computed from it stays behind this point.
__device__ __forceinline__ void reform(uint32_t& v) { asm volatile("" : "+v"(v)); }

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

// Waits until all this wavefront's LDS accesses are done.
__device__ __forceinline__ void wait_lds() {
    __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4));
}

// An operand whose sum index is contiguous in memory: EXT positions (rows or
// features) x 64 elements of the sum, 128 bytes per position. 16-byte chunk c
// of position p sits at chunk c ^ swz(p). A 16-byte LDS read serves 16 lanes at
// a time, lanes 0-3, 12-15, 20-23 and 24-27 of a half wavefront together, then
// the others; with p / 2 % 8 both sets, which hold all 16 positions of a
// fragment at chunks c and c ^ 1, fall into 16 distinct bank groups. A direct
// load writes 64 consecutive chunks, so the swizzle is applied to the address
// each lane reads.
template <int EXT, int WAVES>
struct PackedOperand {
    static constexpr int kChunks = EXT * 8;
    static constexpr int kLoads = EXT / (8 * WAVES);
    static constexpr int kFragReads = 1;
    static_assert(EXT % (8 * WAVES) == 0, "whole wavefront loads");
    const char* base[kLoads];  // wavefront-uniform
    uint32_t off[kLoads];
    int wave;
    uint32_t frag_at;          // byte of this lane's fragment of block blk0, first half

    __device__ static int swz(int p) { return (p >> 1) & 7; }

    // The chunk lane `lane` loads for load j.
    __device__ int chunk_of(int j, int lane) const {
        return (lane & 7) ^ swz((wave + WAVES * j) * 8 + (lane >> 3));
    }
    // row(p) gives the matrix row of position p relative to base_of(p); both
    // are uniform over groups of 8 positions except for the row itself.
    template <class Base, class Row>
    __device__ void init(int wave_, int lane, int blk0, int64_t pitch, Base base_of, Row row) {
        wave = wave_;
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int p0 = (wave + WAVES * j) * 8;
            const int p = p0 + (lane >> 3);
            base[j] = base_of(p0);
            off[j] = static_cast<uint32_t>(row(p) * pitch) + chunk_of(j, lane) * 16;
        }
        const int i = lane & 15, g = lane >> 4;
        frag_at = ((blk0 * 16 + i) * 8 + (g ^ swz(i))) * 16;
    }
    __device__ void issue(int64_t step, v4i* buf) const {
#pragma unroll
        for (int j = 0; j < kLoads; ++j)
            load_to_lds(base[j] + step * 128, off[j],
                        buf + (wave + WAVES * j) * 64);
    }
    // The last, partial step holds `left` (1..63) of the sum. Its loads read
    // something valid past them, which fix() replaces by zeros in LDS.
    __device__ void issue_partial(int64_t step, int left, int lane, v4i* buf) const {
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const uint32_t c = chunk_of(j, lane);
            load_to_lds(base[j] + step * 128,
                        off[j] - (c * 8 < static_cast<uint32_t>(left) ? 0 : c * 16),
                        buf + (wave + WAVES * j) * 64);
        }
    }
    __device__ void fix(int left, int lane, v4i* buf) const {
#pragma unroll
        for (int j = 0; j < kLoads; ++j)
            if (chunk_of(j, lane) * 8 >= left)
                buf[(wave + WAVES * j) * 64 + lane] = v4i{0, 0, 0, 0};
    }
    // Positions [16 (blk0 + b), + 16), half s of the step: chunk 4s + g, so
    // the halves differ in one address bit.
    __device__ bf16x8 frag(const v4i* buf, int b, int s) const {
        const char* p = reinterpret_cast<const char*>(buf) + (frag_at ^ (64 * s)) + b * 2048;
        return __builtin_bit_cast(bf16x8, *reinterpret_cast<const v4i*>(p));
    }
};

// An operand whose sum index strides in memory: a step of ROWS (32 or 64) rows
// of the sum x EXT contiguous positions. Fragments come out of LDS transposed (ds_read_b64_tr:
// a group of 16 lanes reads 4 sum rows of 32 bytes and each lane receives one
// position's 4 elements). The 32-byte blocks of a sum row are stored at block
// b ^ f(row) with f(row) = row % 4 + 4 * (row / 8 % 2): the 8 sum rows two
// lane groups read together then lie in distinct banks.
template <int EXT, int WAVES, int ROWS>
struct StridedOperand {
    static constexpr int kRowChunks = EXT / 8;
    static constexpr int kChunks = ROWS * kRowChunks;
    static constexpr int kLoads = kChunks / (64 * WAVES);
    static constexpr int kFragReads = 2;
    static_assert(EXT % 128 == 0 && kChunks % (64 * WAVES) == 0, "whole wavefront loads");
    const char* base;          // wavefront-uniform
    int64_t step_bytes;
    uint32_t off[kLoads];
    int wave;
    uint32_t frag_at;          // byte of this lane's fragment of block blk0, first half

    __device__ static int fswz(int k) { return (k & 3) | ((k >> 1) & 4); }

    // base_: element (first sum row, first position) of the tile; positions
    // at or past `width` (a multiple of 8) read the last valid chunk. blk0 is
    // a multiple of the number of blocks read from it (a power of two).
    __device__ void init(int wave_, int lane, int blk0, int64_t pitch, const char* base_,
                         int32_t width) {
        wave = wave_;
        base = base_;
        step_bytes = pitch * ROWS;
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int q = (wave + WAVES * j) * 64 + lane;
            const int k = q / kRowChunks, pos = q % kRowChunks;
            const int c = (((pos >> 1) ^ fswz(k)) << 1) | (pos & 1);
            off[j] = static_cast<uint32_t>(k * pitch) + min(c, width / 8 - 1) * 16;
        }
        const int i = lane & 15, g = lane >> 4;
        const int fx = (i >> 2) | ((g & 1) << 2);
        frag_at = (8 * g + (i >> 2)) * (EXT * 2) + (i & 3) * 8 + ((blk0 ^ fx) * 32);
    }
    __device__ void issue(int64_t step, v4i* buf) const {
        const char* at = base + step * step_bytes;
#pragma unroll
        for (int j = 0; j < kLoads; ++j) load_to_lds(at, off[j], buf + (wave + WAVES * j) * 64);
    }
    // The last, partial step holds `left` (fewer) sum rows. The loads past
    // them read its first row, which fix() replaces by zeros in LDS.
    __device__ int row_of(int j, int lane) const {
        return ((wave + WAVES * j) * 64 + lane) / kRowChunks;
    }
    __device__ void issue_partial(int64_t step, int left, int lane, v4i* buf) const {
        const char* at = base + step * step_bytes;
        const uint32_t pitch = static_cast<uint32_t>(step_bytes / ROWS);
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int k = row_of(j, lane);
            load_to_lds(at, off[j] - (k < left ? 0 : k * pitch), buf + (wave + WAVES * j) * 64);
        }
    }
    __device__ void fix(int left, int lane, v4i* buf) const {
#pragma unroll
        for (int j = 0; j < kLoads; ++j)
            if (row_of(j, lane) >= left)
                buf[(wave + WAVES * j) * 64 + lane] = v4i{0, 0, 0, 0};
    }
    __device__ bf16x8 frag(const v4i* buf, int b, int s) const {
        const char* p =
            reinterpret_cast<const char*>(buf) + (frag_at ^ (b * 32)) + s * (32 * EXT * 2);
        const bf16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)(p));
        const bf16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)(p + 4 * EXT * 2));
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
};

// The products of A's 16-position blocks blk0 + a with B's blocks blk0 + b,
// summed over `length` elements in steps of 64. Every wavefront of the
// workgroup calls it.
//
// A step is two halves of 32. While the products of one half run, the LDS reads
// of the next half go out between them, so the matrix cores wait neither for
// LDS nor for memory: the second half is read during the first one's products;
// then every wavefront has read the whole step, and after the step's one
// barrier its buffers take the loads of step + STAGES, and the next step's
// first half is read during the second one's products.
template <int STAGES, int NA, int NB, class A, class B>
struct Accumulator {
    static constexpr int kLoads = A::kLoads + B::kLoads;
    static constexpr int kReads = NA * A::kFragReads + NB * B::kFragReads;  // of a half
    struct Frags {
        bf16x8 a[NA], b[NB];
    };
    // LDS of the stages, each A's part, then B's.
    static constexpr int kStage = A::kChunks + B::kChunks;
    static constexpr int kLdsChunks = STAGES * kStage;
    v4i* lds;
    int lane;
    int32_t first;          // the whole steps are taken from this one on, then from 0
    int32_t whole;          // how many there are

    // Memory step of the t-th whole step.
    __device__ __forceinline__ int32_t at(int32_t t) const {
        t += first;
        return t >= whole ? t - whole : t;
    }
    __device__ static int32_t steps_of(int64_t length) {
        return static_cast<int32_t>((length + 63) / 64);
    }
    // A partial step (length not a multiple of 64) comes first, so that the
    // loop holds whole steps only: step t of the loop is whole step t - 1 then.
    __device__ static int left_of(int64_t length) { return static_cast<int>(length & 63); }
    __device__ __forceinline__ void issue(const A& opa, const B& opb, int stage, int32_t t) const {
        opa.issue(at(t), lds + stage * kStage);
        opb.issue(at(t), lds + stage * kStage + A::kChunks);
    }
    // The first steps' loads.
    __device__ __forceinline__ void start(const A& opa, const B& opb, int64_t length) const {
        const int32_t steps = steps_of(length);
        const int left = left_of(length);
        if (left != 0) {
            opa.issue_partial(steps - 1, left, lane, lds);
            opb.issue_partial(steps - 1, left, lane, lds + A::kChunks);
        } else if (steps > 0) {
            issue(opa, opb, 0, 0);
        }
        const int32_t skip = left != 0 ? 1 : 0;
#pragma unroll
        for (int t = 1; t < STAGES; ++t)
            if (t < steps) issue(opa, opb, t, t - skip);
    }
    __device__ __forceinline__ void fetch_half(const A& opa, const B& opb, int stage, int s,
                                               Frags& d) const {
        // The blocks' addresses are formed here from a register each: what the
        // compiler would form ahead of the loop does not fit the registers.
        A oa = opa;
        B ob = opb;
        reform(oa.frag_at);
        reform(ob.frag_at);
        const v4i* buf = lds + stage * kStage;
#pragma unroll
        for (int a = 0; a < NA; ++a) d.a[a] = oa.frag(buf, a, s);
#pragma unroll
        for (int b = 0; b < NB; ++b) d.b[b] = ob.frag(buf + A::kChunks, b, s);
    }
    // The order within a half: an LDS read after every few products.
    __device__ __forceinline__ static void spread() {
        constexpr int per = NA * NB / kReads > 0 ? NA * NB / kReads : 1;
#pragma unroll
        for (int q = 0; q < kReads; ++q) {
            __builtin_amdgcn_sched_group_barrier(0x008, per, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
    }
    // Sums into acc (cleared first).
    __device__ __forceinline__ void run(const A& opa, const B& opb, int64_t length,
                                        f32x4 (&acc)[NA][NB]) const {
#pragma unroll
        for (int a = 0; a < NA; ++a)
#pragma unroll
            for (int b = 0; b < NB; ++b) acc[a][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        const int32_t steps = steps_of(length);
        const int left = left_of(length);
        if (steps == 0) return;
        const int32_t ahead = left != 0 ? STAGES - 1 : STAGES;
        auto multiply = [&](const Frags& d) {
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int a = 0; a < NA; ++a)
                    acc[a][b] =
                        __builtin_amdgcn_mfma_f32_16x16x32_bf16(d.a[a], d.b[b], acc[a][b], 0, 0, 0);
        };
        Frags lo, hi;
        start(opa, opb, length);
        if (steps < STAGES)
            wait_loads<0>();
        else
            wait_loads<kLoads*(STAGES - 1)>();
        step_barrier();
        if (left != 0) {
            opa.fix(left, lane, lds);
            opb.fix(left, lane, lds + A::kChunks);
            wait_lds();
            step_barrier();
        }
        fetch_half(opa, opb, 0, 0, lo);
        int stage = 0;
        for (int32_t t = 0; t < steps; ++t) {
            fetch_half(opa, opb, stage, 1, hi);
            multiply(lo);
            spread();
            // At most the loads of the steps after the next one are in flight.
            if (STAGES > 2 && t + STAGES - 1 < steps)
                wait_loads<kLoads*(STAGES - 2)>();
            else
                wait_loads<0>();
            step_barrier();
            if (t + STAGES < steps) issue(opa, opb, stage, t + ahead);
            stage = stage + 1 == STAGES ? 0 : stage + 1;
            // After the last step this reads what an earlier one left; it is
            // not used.
            fetch_half(opa, opb, stage, 0, lo);
            multiply(hi);
            spread();
        }
    }
};

// act(g) and its derivative in fp32. silu(g) = g sigmoid(g); the tanh form of
// gelu is g sigmoid(2z) with z = sqrt(2/pi) (g + 0.044715 g^3), which loses no
// digits where 1 + tanh(z) would cancel. exp runs to infinity or zero at the
// ends, where the sigmoid is exactly 0 or 1; one below 2^-126 (silu from g = -87.4
// down, gelu from -10.0) becomes 0 too, since the reciprocal returns no denormals.
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

// Rounded to nearest even (a NaN stays one), element 2i in the low half.
__device__ __forceinline__ v2i pack_bf16x4(f32x4 v) {
    return __builtin_bit_cast(v2i, __builtin_convertvector(v, bf16x4));
}

// A register of which lane group g holds value g of the 16 lanes' to four
// registers that hold value 0, 1, 2 and 3 in all groups.
__device__ __forceinline__ void spread(uint32_t v, uint32_t (&d)[4]) {
    const auto half = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    const auto lo = __builtin_amdgcn_permlane16_swap(half[0], half[0], false, false);
    const auto hi = __builtin_amdgcn_permlane16_swap(half[1], half[1], false, false);
    d[0] = lo[0];
    d[1] = lo[1];
    d[2] = hi[0];
    d[3] = hi[1];
}

// Four bf16 of block a and of the next block per lane (lane group g holds
// elements 4g .. 4g + 3 of each, of one row), exchanged between groups 0 and 1
// and between 2 and 3 so that every lane holds eight neighbours: elements
// 8 (g / 2) .. + 8 of block a + g % 2. Stores then take half as many
// instructions and cover 64 contiguous bytes of a row instead of 32.
__device__ __forceinline__ v4i pair_blocks(v2i a, v2i b) {
    const auto lo = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    const auto hi = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    return v4i{static_cast<int32_t>(lo[0]), static_cast<int32_t>(hi[0]),
               static_cast<int32_t>(lo[1]), static_cast<int32_t>(hi[1])};
}

}  // namespace moe
