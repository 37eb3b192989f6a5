// Gradient of the expert weights on gfx950: for every expert e
//     dw[e][n][k] = sum over rows r of e's segment of dy[r][n] * x[r][k]
// (plus what dw holds, on request), one rounding of the fp32 sum.
//
// Both operands stride along the sum (the rows), which the matrix cores want
// contiguous: LDS is read transposed. A workgroup owns a tile of one expert's
// gradient and walks its rows, so no sum is shared between workgroups, nothing
// is joined afterwards and the order of a sum is the rows' order.
//
// Bound. The gradient is written once, and a segment of c rows gives c operations
// per byte of it in bf16: its bytes count up to some 200 rows per expert, the
// matrix cores above. 128 x 256 of four wavefronts, two workgroups to a CU: one
// fills its first stages or writes its results while the other multiplies. Tried
// at 512 rows per expert, 4096 x 4096: 256 x 256 with steps of 64 rows, one to a
// CU, 3.13 against 2.84 ms; 128 x 128, three to a CU, 2.96 against 2.74 (at 128
// rows and 2048 x 1408, which 128 divides better, 189 against 212 us; at 2816 x
// 2048 378 against 366); workgroups that stay and load the next tile early, 3.5.
//
// Measured on MI355X (a large library product reaches 1438 TFLOP/s), behind other
// products as in a training step: 128 experts of 512 rows on average, routed at
// random, 4096 x 2048 1.31 to 1.32 ms (0.83 PFLOP/s), 4096 x 4096 2.58 to 2.60 ms
// (0.85); of 128 rows, 2048 x 1408 241 to 259 us, 2816 x 2048 420 to 484 us. Exactly
// 512 rows per expert, by themselves: 1.24 and 2.51 ms where routed rows take 1.31
// and 2.62. One expert of 65536 rows: 1.23 to 1.31 PFLOP/s. LDS bank conflicts
// count 0.
//
// fp32 gradients are twice the bytes: 4096 x 4096 routed 3.29 ms against 2.70 in
// bf16, 2816 x 2048 (128 rows on average) 0.51 against 0.41 ms. Adding reads the
// gradient as well, and its lanes write pieces of 4 values where the other forms
// write whole rows: 4.2 ms (bf16) and 5.1 ms (fp32), 1.07 and 1.33 ms.
#include "expert_kernels.h"
#include "expert_mma.h"

namespace moe {
namespace {

constexpr int kWaves = 4;
constexpr int kWavesK = 2;
constexpr int kWavesN = 2;
constexpr int kTileK = 256;
constexpr int kTileN = 128;
constexpr int kBlkK = kTileK / kWavesK / 16;
constexpr int kBlkN = kTileN / kWavesN / 16;
constexpr int kStep = 32;               // rows per step: one matrix-core product deep
constexpr int kStages = 3;              // 72 KiB of LDS: two workgroups per CU
constexpr int kXcdChunk = 64;
constexpr int kTouch = 16;              // workgroups that touch one expert's rows

typedef StridedOperand<kTileK, kWaves, kStep> Kop;
typedef StridedOperand<kTileN, kWaves, kStep> Nop;
constexpr int kLoads = Kop::kLoads + Nop::kLoads;
constexpr int kStageChunks = Kop::kChunks + Nop::kChunks;

struct Frags {
    bf16x8 k[kBlkK], n[kBlkN];
};

__device__ __forceinline__ void fetch(const Kop& ko, const Nop& no, const v4i* buf, Frags& d) {
    // The blocks' addresses are formed here from a register each: what the
    // compiler would form ahead of the loop does not fit the registers.
    Kop kk = ko;
    Nop nn = no;
    reform(kk.frag_at);
    reform(nn.frag_at);
#pragma unroll
    for (int a = 0; a < kBlkK; ++a) d.k[a] = kk.frag(buf, a, 0);
#pragma unroll
    for (int b = 0; b < kBlkN; ++b) d.n[b] = nn.frag(buf + Kop::kChunks, b, 0);
}

// A tile's results on their way out through LDS: rows of CHUNKS 16-byte chunks,
// chunk c of row r at c ^ (r % 16), so that writes of one chunk of 16 rows and
// reads of whole rows both spread over the banks. From there whole rows go out,
// CHUNKS * 16 contiguous bytes each; from the products' own lanes they would
// leave in pieces of 64 bytes. Streamed past the caches: the gradient is as
// large as the weights and is not read here.
template <int ROWS, int CHUNKS>
struct OutTile {
    __device__ static int at(int row, int chunk) { return row * CHUNKS + (chunk ^ (row & 15)); }
    // Rows [0, rows) to dst, `pitch` bytes apart, their first `chunks` chunks.
    __device__ __forceinline__ static void store(const v4i* lds, char* dst, int64_t pitch,
                                                 int rows, int chunks, int wave, int lane) {
        constexpr int kRows = 64 / CHUNKS;          // of one store
        const int c = lane % CHUNKS;
        const int r0 = wave * (ROWS / kWaves) + lane / CHUNKS;
#pragma unroll
        for (int q = 0; q < ROWS / kWaves / kRows; ++q) {
            const int r = r0 + q * kRows;
            const v4i v = lds[at(r, c)];
            if (r < rows && c < chunks)
                __builtin_nontemporal_store(v, reinterpret_cast<v4i*>(dst + r * pitch) + c);
        }
    }
};

// Reads part `part` of kTouch of `bytes` (whole 16-byte chunks) and drops them:
// they are in the memory-side cache then.
__device__ __forceinline__ void touch_rows(const char* base, int64_t bytes, int part) {
    constexpr int kThreads = kWaves * 64, kAtOnce = 8;
    const v4i* p = reinterpret_cast<const v4i*>(base);
    const int64_t chunks = bytes / 16, end = chunks * (part + 1) / kTouch;
    int64_t i = chunks * part / kTouch + threadIdx.x;
    int32_t seen = 0;
    for (; i + (kAtOnce - 1) * kThreads < end; i += kAtOnce * kThreads) {
        v4i v[kAtOnce];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) v[j] = p[i + j * kThreads];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) seen ^= v[j][0];
    }
    for (; i < end; i += kThreads) seen ^= p[i][0];
    asm volatile("" ::"v"(seen));       // the loads have a use
}

// The launch's workgroups, in the order they start. With touch != 0 (kTouch):
// first the ones that touch the rows of experts 0 .. ahead - 1, then for every
// expert those that touch the rows of the expert `ahead` later, and its tiles.
template <bool F32, bool ACCUMULATE>
__global__ __launch_bounds__(kWaves * 64, 2)
void expert_wgrad_kernel(const char* __restrict__ dy, const char* __restrict__ x,
                         const int32_t* __restrict__ offsets, int32_t max_rows, int32_t N,
                         int32_t K, int32_t ntiles, int32_t ktiles, int32_t E, int32_t touch,
                         int32_t ahead, int64_t jobs, char* __restrict__ dw) {
    __shared__ v4i lds[kStages * kStageChunks];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int64_t u = expert_tile_number(kXcdChunk);
    if (u >= jobs) return;
    const int64_t front = int64_t(touch) * ahead;
    int32_t e, in;
    if (u < front) {
        e = static_cast<int32_t>(u / touch);
        in = static_cast<int32_t>(u - int64_t(e) * touch);
    } else {
        const int32_t per = touch + ntiles * ktiles;
        u -= front;
        e = static_cast<int32_t>(u / per);
        in = static_cast<int32_t>(u - int64_t(e) * per);
        if (in < touch) e += ahead;
    }
    if (e >= E) return;
    int32_t s0, s1;
    expert_segment(offsets, e, max_rows, s0, s1);
    const int32_t count = s1 - s0;
    if (in < touch) {
        touch_rows(x + int64_t(s0) * K * 2, int64_t(count) * K * 2, in);
        touch_rows(dy + int64_t(s0) * N * 2, int64_t(count) * N * 2, in);
        return;
    }
    in -= touch;
    if (ACCUMULATE && count == 0) return;
    // Tiles along K first where a segment is short: what runs at once then
    // writes long contiguous pieces of dw. From 2048 rows on the rows' reads
    // weigh more, and bands of 8 tiles along N share them in the L2 cache.
    const int32_t deep = count >= 2048 ? 8 : 1;
    const int32_t band = in / (ktiles * deep);
    const int32_t inside = in - band * ktiles * deep;
    const int32_t height = min(deep, ntiles - band * deep);
    const int32_t nt0 = (band * deep + inside % height) * kTileN;
    const int32_t kt0 = inside / height * kTileK;

    Kop ko;
    Nop no;
    const int wk = wave % kWavesK, wn = wave / kWavesK;
    ko.init(wave, lane, wk * kBlkK, int64_t(K) * 2, x + (int64_t(s0) * K + kt0) * 2,
            min(kTileK, K - kt0));
    no.init(wave, lane, wn * kBlkN, int64_t(N) * 2, dy + (int64_t(s0) * N + nt0) * 2,
            min(kTileN, N - nt0));
    f32x4 acc[kBlkK][kBlkN];
#pragma unroll
    for (int a = 0; a < kBlkK; ++a)
#pragma unroll
        for (int b = 0; b < kBlkN; ++b) acc[a][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    const int32_t steps = expert_row_parts(count, kStep);
    if (steps > 0) {
        auto issue = [&](int stage, int32_t t) {
            ko.issue(t, lds + stage * kStageChunks);
            no.issue(t, lds + stage * kStageChunks + Kop::kChunks);
        };
        // A partial step comes first, so that the loop holds whole steps only:
        // step t of the loop is step t - 1 of memory then.
        const int left = count % kStep;
        const int32_t skip = left != 0 ? 1 : 0;
        if (left != 0) {
            ko.issue_partial(steps - 1, left, lane, lds);
            no.issue_partial(steps - 1, left, lane, lds + Kop::kChunks);
        } else {
            issue(0, 0);
        }
#pragma unroll
        for (int t = 1; t < kStages; ++t)
            if (t < steps) issue(t, t - skip);
        if (steps < kStages)
            wait_loads<0>();
        else
            wait_loads<kLoads*(kStages - 1)>();
        step_barrier();
        if (left != 0) {
            ko.fix(left, lane, lds);
            no.fix(left, lane, lds + Kop::kChunks);
            wait_lds();
            step_barrier();
        }
        Frags even, odd;
        fetch(ko, no, lds, even);
        int stage = 0;
        // Products of one step, while the next one's fragments are read.
        auto step = [&](const Frags& now, Frags& next, int32_t t) {
            // The next step has landed (at most the loads of those after it
            // are in flight) and this one's reads have returned.
            if (t + kStages - 1 < steps)
                wait_loads<kLoads*(kStages - 2)>();
            else
                wait_loads<0>();
            step_barrier();
            if (t + kStages < steps) issue(stage, t + kStages - skip);
            stage = stage + 1 == kStages ? 0 : stage + 1;
            // After the last step this reads what an earlier one left; it is
            // not used.
            fetch(ko, no, lds + stage * kStageChunks, next);
#pragma unroll
            for (int b = 0; b < kBlkN; ++b)
#pragma unroll
                for (int a = 0; a < kBlkK; ++a)
                    acc[a][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(now.k[a], now.n[b],
                                                                        acc[a][b], 0, 0, 0);
            // An LDS read (two to a fragment) after each product.
#pragma unroll
            for (int q = 0; q < 2 * (kBlkK + kBlkN); ++q) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
        };
        // Two steps a turn; an odd number ends with a step of zeros.
        for (int32_t t = 0; t < steps; t += 2) {
            step(even, odd, t);
            if (t + 1 >= steps) {
#pragma unroll
                for (int a = 0; a < kBlkK; ++a) odd.k[a] = bf16x8{};
#pragma unroll
                for (int b = 0; b < kBlkN; ++b) odd.n[b] = bf16x8{};
            }
            step(odd, even, t + 1);
        }
    }

    const int i = lane & 15, g = lane >> 4;
    char* tile = dw + ((int64_t(e) * N + nt0) * K + kt0) * (F32 ? 4 : 2);
    const int rows = min(kTileN, N - nt0), width = min(kTileK, K - kt0);
    if constexpr (ACCUMULATE) {
        // Every lane adds to four neighbours of one row.
#pragma unroll
        for (int b = 0; b < kBlkN; ++b) {
            const int n = (wn * kBlkN + b) * 16 + i;
            if (n >= rows) continue;
#pragma unroll
            for (int a = 0; a < kBlkK; ++a) {
                const int k = (wk * kBlkK + a) * 16 + g * 4;
                if (k >= width) continue;
                char* at = tile + (int64_t(n) * K + k) * (F32 ? 4 : 2);
                f32x4 v = acc[a][b];
                if constexpr (F32) {
                    f32x4* p = reinterpret_cast<f32x4*>(at);
                    *p = *p + v;
                } else {
                    v2i* p = reinterpret_cast<v2i*>(at);
                    const v2i o = *p;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint32_t word = static_cast<uint32_t>(o[q >> 1]);
                        v[q] += (q & 1) ? bf16_hi(word) : bf16_lo(word);
                    }
                    *p = pack_bf16x4(v);
                }
            }
        }
    } else if constexpr (F32) {
        // 64 KiB at a time: the rows of half the blocks, then of the others.
        typedef OutTile<kBlkN / 2 * 16, kTileK / 4> Out;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            if (half) __syncthreads();
#pragma unroll
            for (int b = 0; b < kBlkN / 2; ++b)
#pragma unroll
                for (int a = 0; a < kBlkK; ++a)
                    lds[Out::at((wn * (kBlkN / 2) + b) * 16 + i, (wk * kBlkK + a) * 4 + g)] =
                        __builtin_bit_cast(v4i, acc[a][half * (kBlkN / 2) + b]);
            __syncthreads();
#pragma unroll
            for (int p = 0; p < kWavesN; ++p) {
                const int first = (p * kBlkN + half * (kBlkN / 2)) * 16;
                Out::store(lds + p * (kBlkN / 2) * 16 * (kTileK / 4),
                           tile + int64_t(first) * K * 4, int64_t(K) * 4, rows - first, width / 4,
                           wave, lane);
            }
        }
    } else {
        typedef OutTile<kTileN, kTileK / 8> Out;
#pragma unroll
        for (int b = 0; b < kBlkN; ++b)
#pragma unroll
            for (int a = 0; a < kBlkK; a += 2)
                lds[Out::at((wn * kBlkN + b) * 16 + i, (wk * kBlkK + a + (g & 1)) * 2 + (g >> 1))] =
                    pair_blocks(pack_bf16x4(acc[a][b]), pack_bf16x4(acc[a + 1][b]));
        __syncthreads();
        Out::store(lds, tile, int64_t(K) * 2, rows, width / 8, wave, lane);
    }
}

int32_t k_tiles(const ExpertWgradArgs& a) {
    return static_cast<int32_t>((int64_t(a.K) + kTileK - 1) / kTileK);
}
int32_t n_tiles(const ExpertWgradArgs& a) {
    return static_cast<int32_t>((int64_t(a.N) + kTileN - 1) / kTileN);
}
int64_t tiles_per_expert(const ExpertWgradArgs& a) { return int64_t(n_tiles(a)) * k_tiles(a); }

// Whether rows are touched ahead of their tiles. A tile of a short segment is
// little more than the latency of its reads, and where the rows are not in the
// memory-side cache (another product has run since they were written) those
// queue behind the gradient's own writes. Measured on MI355X behind a product of
// other weights: 128 experts of 128 rows, 2048 x 1408, 296 us without and 241
// with it, 2816 x 2048 490 and 420; 16 such experts 63.9 and 53.8; 256 of 8 rows,
// 2048 x 7168, 1481 and 1239; 128 of 512 rows, 4096 x 2048 1400 and 1305, 4096 x
// 4096 2801 and 2581. Longer segments read ahead in their own loops: 32 of 1024
// rows, 4096 x 4096, 1070 and 1106, 16 of 4096 rows 1709 and 1880. Repeated on
// rows that are in the cache it costs 3 to 6 % (128 rows: 212 and 219, 366 and
// 389). 32 workgroups per expert instead of 16 lose at 2048 x 1408 (306).
// Not where an expert has few tiles beside the 16 workgroups (256 experts of 64
// rows: 256 x 512, 4 tiles, 25.3 and 32.8 us; 512 x 1024, 16 tiles, 77.2 and 74.7;
// 1024 x 1024, 32 tiles, 153 and 132), nor where all tiles start at once anyway
// (one expert of 256 rows, 4096 x 4096, 512 tiles, 17.3 and 23.0 us; 8 of 128 rows,
// 2816 x 2048, 1408 tiles, 33.6 and 32.2).
bool touches(const ExpertWgradArgs& a) {
    return a.max_rows <= int64_t(512) * a.E && tiles_per_expert(a) >= kTouch &&
           tiles_per_expert(a) * a.E >= 1024;
}

// How many experts ahead: all at once if the rows fit the memory-side cache (256
// MB) with room for others, else what one or two rounds of workgroups take
// (128 experts of 128 rows, one to two rounds ahead: 283 and 479 us). At 512
// rows 2048 tiles ahead are as good as 1024, 8192 lose 5 %.
int32_t touched_ahead(const ExpertWgradArgs& a) {
    if (a.max_rows * (int64_t(a.N) + a.K) * 2 <= (int64_t(192) << 20)) return a.E;
    const int64_t per = tiles_per_expert(a);
    const int64_t ahead = (1024 + per - 1) / per;
    return static_cast<int32_t>(ahead < a.E ? ahead : a.E);
}
int64_t job_count(const ExpertWgradArgs& a) {
    const int64_t touch = touches(a) ? kTouch : 0;
    return (tiles_per_expert(a) + touch) * a.E + touch * touched_ahead(a);
}

int64_t grid_of(const ExpertWgradArgs& a) {
    const int64_t unit = int64_t(kExpertXcds) * kXcdChunk;
    return (job_count(a) + unit - 1) / unit * unit;
}

}  // namespace

int64_t expert_wgrad_grid(const ExpertWgradArgs& a) { return grid_of(a) * (kWaves * 64); }

hipError_t launch_expert_wgrad(const ExpertWgradArgs& a, hipStream_t stream) {
    auto kernel = a.f32 ? (a.accumulate ? expert_wgrad_kernel<true, true>
                                        : expert_wgrad_kernel<true, false>)
                        : (a.accumulate ? expert_wgrad_kernel<false, true>
                                        : expert_wgrad_kernel<false, false>);
    hipLaunchKernelGGL(kernel, dim3(static_cast<uint32_t>(grid_of(a))),
                       dim3(kWaves * 64), 0, stream, static_cast<const char*>(a.dy),
                       static_cast<const char*>(a.x), a.offsets, static_cast<int32_t>(a.max_rows),
                       a.N, a.K, n_tiles(a), k_tiles(a), a.E, touches(a) ? kTouch : 0,
                       touched_ahead(a), job_count(a), static_cast<char*>(a.dw));
    return hipGetLastError();
}

}  // namespace moe
