// The kernel of the dense product for more than a few rows: tiles of rows of x times rows of w, through LDS, on the
// matrix instructions. Included by one source file per pair of types.
//
// A step is kBK values of k. While one is multiplied the next ones go from memory straight to LDS, into two to four buffers.
// A float32 operand goes through registers, where each value is split into three bfloat16 whose sum is the value (each the
// rounded rest of the ones before: 8 + 8 + 8 bits of a float32's 24). A bfloat16 times a float32 value is then three exact
// products, two float32 values take the six of the nine that reach 2^-23 of the product. That is float32's precision at a
// third (a sixth) of the bfloat16 rate; the float32 matrix instructions have a sixteenth.
//
// What bounds it, with the chip full: the matrix instructions and the loads' way into LDS, which do not overlap all the time
// (the matrix unit is busy for half of it). A step of a 256 x 256 bfloat16 tile is 64 KiB in and 8.4 MFLOP. Measured, fastest
// and median of a graph of calls (the chip slows down while they follow one another):
//   bfloat16 x bfloat16  8192 x 8192 x 8192 813-831 us (1.32-1.35 PFLOP/s); 8192 x 4096 x 4096 215-226, with bias, SiLU and
//                        residual 233-245
//   bfloat16 x float32   8192 x 4096 x 4096 602-621 us (1.33-1.37 PFLOP/s of the three products)
//   float32 x bfloat16   8192 x 4096 x 4096 620-645 us (1.28-1.33)
//   float32 x float32    4096 x 4096 x 4096 564-583 us (1.41-1.46 PFLOP/s of the six)
// Smaller products are bound by what a step takes on a CU with little of its own work: the trip to LDS and the barrier.
#pragma once

#include <type_traits>

#include "lds_loads.h"
#include "linear_common.h"

namespace moed {

// Where a call's tiles lie. splits > 1: each split's sums go to partial [splits][B][N] instead of the epilogue.
struct LinearPlan {
    float* partial;
    int n_blocks, m_blocks, splits, split_steps;
    int group;              // blocks of w's rows that are taken together
};

namespace {

// One operand's rows of a tile: where a thread's part of them comes from and where it lies in LDS.
// In LDS a row of a step is BK bfloat16, U units of 16 bytes; a float32 operand has three such planes, its parts. A
// bfloat16 operand whose rows begin at dwords (DIRECT) goes there straight from memory; otherwise a step's values are
// fetched to registers while the steps before it are multiplied, and put there (float32: split) behind that. Either way
// a thread takes 16 bytes of a row, and its neighbours the next.
template <bool F32, bool DIRECT, int ROWS, int THREADS, int BK>
struct LinearSide {
    static constexpr bool kDirect = DIRECT && !F32;
    static constexpr int kParts = F32 ? 3 : 1, U = BK / 8;
    static constexpr int kPlane = ROWS * U * 16, kBytes = kParts * kPlane;
    static constexpr int kAcross = F32 ? 2 * U : U;           // threads of a row
    static constexpr int kChunks = ROWS * kAcross / THREADS;  // of 16 bytes, a thread and step
    static constexpr int kFetches = kDirect ? 0 : kChunks;
    static_assert(ROWS * kAcross % THREADS == 0 && THREADS / kAcross % 16 == 0, "whole chunks, which share their place in the row");

    const uint8_t* base;
    uint32_t off[kChunks];                                    // of this thread's rows
    int unit, place;                                          // in the row: in memory, and the byte in LDS
    u32x4 held[2][kChunks];                                   // two steps' values on their way

    // rows behind `last` repeat it
    __device__ __forceinline__ void init(const void* p, size_t row0, int last, int K, int tid)
    {
        const size_t row = (size_t)K * (F32 ? 4 : 2);
        base = static_cast<const uint8_t*>(p) + row0 * row;
        const int t = tid % kAcross, swizzle = linear_swizzle<U>(tid / kAcross);
        unit = F32 ? t : t ^ swizzle;                         // straight to LDS: thread t's bytes land at unit t
        place = F32 ? ((t / 2) ^ swizzle) * 16 + (t & 1) * 8 : t * 16;
        place += tid / kAcross * (U * 16);
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            const int r = i * (THREADS / kAcross) + tid / kAcross;
            off[i] = (uint32_t)(r < last ? r : last) * (uint32_t)row;
        }
    }
    __device__ __forceinline__ void load(int st, uint32_t to, int w) const
    {
        const uint8_t* from = base + (size_t)st * (U * 16);
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
            load_to_lds16(from, off[i] + 16u * unit,
                          (uint32_t)__builtin_amdgcn_readfirstlane((int)(to + (uint32_t)(i * THREADS + w * kWave) * 16u)));
    }
    __device__ __forceinline__ void fetch(int set, int st, int K)
    {
        const int k = st * BK + unit * (F32 ? 4 : 8);
        if ((st + 1) * BK <= K) {
#pragma unroll
            for (int i = 0; i < kChunks; ++i)
                held[set][i] = row_unit_at<F32>(base + off[i], k);
        } else {
#pragma unroll
            for (int i = 0; i < kChunks; ++i)
                held[set][i] = row_unit<F32>(base + off[i], k, K);
        }
    }
    __device__ __forceinline__ void put(int set, uint8_t* to) const
    {
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            uint8_t* at = to + place + i * (THREADS / kAcross) * (U * 16);
            if constexpr (F32) {
                u32x2 part[3];
                split3(held[set][i], part);
#pragma unroll
                for (int q = 0; q < 3; ++q)
                    *reinterpret_cast<u32x2*>(at + q * kPlane) = part[q];
            } else {
                *reinterpret_cast<u32x4*>(at) = held[set][i];
            }
        }
    }
    // The fragment of the 16 rows from `row` on, for k 32 s .. 32 s + 31 of the step: lane group g has 8 of them.
    __device__ __forceinline__ static void fragment(const uint8_t* from, int row, int s, int g, int col, bf16x8 (&part)[kParts])
    {
#pragma unroll
        for (int q = 0; q < kParts; ++q)
            part[q] = __builtin_bit_cast(bf16x8, lds16(from + q * kPlane + row * (U * 16) + linear_unit<U>(col, 4 * s + g)));
    }
};

// In the place of a number of buffers: three of x and two of w.
constexpr int kDeep = 0;

template <bool XF32, bool WF32, bool DIRECT, int RT, int NT, int WR, int WN, int RING, int BK>
struct LinearShape {
    static constexpr int kWaves = WR * WN, kThreads = kWaves * kWave;
    static constexpr int kBM = 16 * RT * WR, kBN = 16 * NT * WN;          // rows of x and of w in a tile
    static constexpr int kBK = BK;
    using X = LinearSide<XF32, DIRECT, kBM, kThreads, kBK>;
    using W = LinearSide<WF32, DIRECT, kBN, kThreads, kBK>;
    static constexpr int kBuffer = X::kBytes + W::kBytes;
    static constexpr int kLds = RING == kDeep ? 3 * X::kBytes + 2 * W::kBytes : RING * kBuffer;
    // outputs of a wavefront on their way out: strips of 16 rows, as many as fit
    static constexpr int kOutRow = 16 * NT + 4;                           // float32 values, padded
    static constexpr int kStrip = kWaves * 16 * kOutRow * 4;
    static constexpr int kStrips = RT * kStrip <= kLds ? RT : RT / 2 * kStrip <= kLds ? RT / 2 : RT / 4;
    static_assert(kStrips >= 1 && kStrips * kStrip <= kLds && kLds <= 163840, "room");
};

}  // namespace

// DIRECT: no bfloat16 rows of odd K.
template <bool XF32, bool WF32, bool DIRECT, int RT, int NT, int WR, int WN, int RING, int BK>
__global__ void __launch_bounds__(WR * WN * kWave)
moe_linear_tiled_kernel(LinearArgs p, LinearPlan plan)
{
    using S = LinearShape<XF32, WF32, DIRECT, RT, NT, WR, WN, RING, BK>;
    using X = typename S::X;
    using W = typename S::W;
    extern __shared__ __align__(16) uint8_t lds[];
    const int tid = threadIdx.x, lane = tid % kWave;
    const int w = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int g = lane / 16, col = lane % 16;
    const int wr = w / WN, wn = w % WN;
    const uint32_t lds0 = (uint32_t)(size_t)(__attribute__((address_space(3))) uint8_t*)lds;

    // neighbouring workgroups of an XCD share rows of x and of w
    const int tiles = plan.n_blocks * plan.m_blocks;
    const int item = xcd_contiguous(blockIdx.x, gridDim.x);
    const int split = item / tiles, tile = item - split * tiles;
    const int first = tile / (plan.group * plan.m_blocks) * plan.group;       // of this group's blocks
    const int rest = tile - first * plan.m_blocks;
    const int width = plan.n_blocks - first < plan.group ? plan.n_blocks - first : plan.group;
    const int mb = rest / width, nb = first + rest - mb * width;
    const size_t m0 = (size_t)mb * S::kBM;
    const int n0 = nb * S::kBN;
    const int all = (p.K + S::kBK - 1) / S::kBK;
    const int st0 = split * plan.split_steps, st1 = st0 + plan.split_steps < all ? st0 + plan.split_steps : all;
    const int full = p.K / S::kBK;                            // steps that do not end behind K

    X x;
    W v;
    x.init(p.x, m0, (size_t)p.B - m0 < (size_t)S::kBM ? (int)((size_t)p.B - m0) - 1 : S::kBM - 1, p.K, tid);
    v.init(p.w, (size_t)n0, p.N - n0 < S::kBN ? p.N - n0 - 1 : S::kBN - 1, p.K, tid);
    // Step st (a whole one) of the operands that go to LDS directly.
    auto load = [&](int st, int buffer) {
        const uint32_t at = lds0 + (uint32_t)(buffer * S::kBuffer);
        if constexpr (X::kDirect)
            x.load(st, at, w);
        if constexpr (W::kDirect)
            v.load(st, at + X::kBytes, w);
    };
    // The same of the others.
    auto fetch = [&](int set, int st) {
        if constexpr (!X::kDirect)
            x.fetch(set, st, p.K);
        if constexpr (!W::kDirect)
            v.fetch(set, st, p.K);
    };
    auto put = [&](int set, int buffer) {
        uint8_t* const to = lds + buffer * S::kBuffer;
        if constexpr (!X::kDirect)
            x.put(set, to);
        if constexpr (!W::kDirect)
            v.put(set, to + X::kBytes);
    };

    f32x4 acc[RT][NT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int f = 0; f < NT; ++f)
            acc[r][f] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    auto compute = [&](int buffer, int s) {
        const uint8_t* xb = lds + buffer * S::kBuffer;
        const uint8_t* wb = xb + X::kBytes;
        bf16x8 wv[NT][W::kParts];
#pragma unroll
        for (int f = 0; f < NT; ++f)
            W::fragment(wb, (wn * NT + f) * 16, s, g, col, wv[f]);
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            bf16x8 xv[X::kParts];
            X::fragment(xb, (wr * RT + r) * 16, s, g, col, xv);
            // small parts first, and the same accumulator not twice in a row
#pragma unroll
            for (int q = (XF32 || WF32) ? 2 : 0; q >= 0; --q)
#pragma unroll
                for (int i = 0; i < X::kParts; ++i)
                    if (q - i >= 0 && q - i < W::kParts)
#pragma unroll
                        for (int f = 0; f < NT; ++f)
                            acc[r][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv[f][q - i], xv[i], acc[r][f], 0, 0, 0);
        }
    };
    constexpr int kLoads = (X::kDirect ? X::kChunks : 0) + (W::kDirect ? W::kChunks : 0);
    if constexpr (X::kDirect && W::kDirect && RING == kDeep) {
        // The largest tiles: 64 KiB a step, which take nearly as long to come as to be multiplied and whose latency two
        // whole buffers cannot cover (8192 x 4096 x 4096: 190 us without loads, 206 with nothing else, 248 together). A
        // wavefront has its fragments of w of a whole step in registers when it has multiplied half of it, so that buffer
        // is then free for the step after the next; x has a third one. Loads are on their way for one and a half and two
        // steps: 219 us. Fragments of x are read two turns of NT matrix instructions ahead of their use, those of w for
        // the step's second half under the first; without the fences the compiler reads them as late as it can (225
        // instead of 214 us). One barrier a step, the first fragments of the next one read under the last turns and all
        // loads issued together behind it, takes 234.
        static_assert(S::kBK == 64 && RT >= NT + 2, "two halves of a step; of x at least two reads behind the last of w");
        uint8_t* const wlds = lds + 3 * X::kBytes;
        const int end = st1 < full ? st1 : full;
        auto load_x = [&](int st, int buffer) { x.load(st, lds0 + (uint32_t)(buffer * X::kBytes), w); };
        auto load_w = [&](int st) { v.load(st, lds0 + (uint32_t)(3 * X::kBytes + (st & 1) * W::kBytes), w); };
        bf16x8 wv[2][NT], xv[4];
        auto read_x = [&](const uint8_t* from, int turn) {
            bf16x8 part[1];
            X::fragment(from, (wr * RT + turn % RT) * 16, turn / RT, g, col, part);
            xv[turn % 4] = part[0];
        };
        auto read_w = [&](const uint8_t* from, int s, int f) {
            bf16x8 part[1];
            W::fragment(from, (wn * NT + f) * 16, s, g, col, part);
            wv[s][f] = part[0];
        };
        auto turn_products = [&](int turn) {
#pragma unroll
            for (int f = 0; f < NT; ++f)
                acc[turn % RT][f] =
                    __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv[turn / RT][f], xv[turn % 4], acc[turn % RT][f], 0, 0, 0);
        };
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (st0 + i < end) {
                load_x(st0 + i, i);
                load_w(st0 + i);
            }
        int buffer = 0;
        for (int st = st0; st < end; ++st) {
            if (st + 1 < end)
                wait_loads<X::kChunks + W::kChunks>();
            else
                wait_loads<0>();
            __syncthreads();                                  // step st is in LDS, and nobody reads the x before it
            if (st + 2 < end)
                load_x(st + 2, buffer == 0 ? 2 : buffer - 1);
            const uint8_t* const xb = lds + buffer * X::kBytes;
            const uint8_t* const wb = wlds + (st & 1) * W::kBytes;
            read_w(wb, 0, 0);
            read_x(xb, 0);
#pragma unroll
            for (int f = 1; f < NT; ++f)
                read_w(wb, 0, f);
            read_x(xb, 1);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int turn = 0; turn < 2 * RT; ++turn) {
                if (turn + 2 < 2 * RT)
                    read_x(xb, turn + 2);
                if (turn < NT)
                    read_w(wb, 1, turn);
                __builtin_amdgcn_sched_barrier(0);
                turn_products(turn);
                __builtin_amdgcn_sched_barrier(0);
                if (turn == RT - 1) {
                    wait_lds<2>();                            // all of w: of what was asked for later, two of x are left
                    barrier();                                // everybody has the step's w
                    if (st + 2 < end)
                        load_w(st + 2);
                }
            }
            buffer = buffer == 2 ? 0 : buffer + 1;
        }
        if (st1 > full) {                                     // zeros behind K
            __syncthreads();
            x.fetch(0, full, p.K);
            v.fetch(0, full, p.K);
            x.put(0, lds);
            v.put(0, wlds);
            __syncthreads();
#pragma unroll
            for (int turn = 0; turn < 2 * RT; ++turn) {
                if (turn % RT == 0)
#pragma unroll
                    for (int f = 0; f < NT; ++f)
                        read_w(wlds, turn / RT, f);
                read_x(lds, turn);
                turn_products(turn);
            }
        }
    } else if constexpr (X::kDirect && W::kDirect) {
        constexpr int kAhead = RING - 1;
        const int end = st1 < full ? st1 : full;
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (st0 + i < end)
                load(st0 + i, i);
        int buffer = 0;
        for (int st = st0; st < end; ++st) {
            // the steps behind this one may be on their way
            if (st + kAhead <= end)
                wait_loads<(kAhead - 1) * kLoads>();
            else
                wait_loads<0>();
            __syncthreads();                                  // step st is in LDS, and nobody reads the one before
            if (st + kAhead < end)
                load(st + kAhead, buffer == 0 ? kAhead : buffer - 1);
            compute(buffer, 0);
            compute(buffer, 1);
            buffer = buffer + 1 == RING ? 0 : buffer + 1;
        }
        if (st1 > full) {                                     // zeros behind K
            __syncthreads();
            x.fetch(0, full, p.K);
            v.fetch(0, full, p.K);
            x.put(0, lds);
            v.put(0, lds + X::kBytes);
            __syncthreads();
            compute(0, 0);
            compute(0, 1);
        }
    } else {
        // Two buffers. While step st is multiplied, step st + 1 comes out of its registers, which then wait for st + 3.
        static_assert(RING == 2, "an operand that goes through registers has two sets of them and two buffers");
        // what goes straight to LDS; zeros behind K by way of registers
        auto load_or_put = [&](int st, int buffer) {
            if (st < full) {
                load(st, buffer);
            } else {
                if constexpr (X::kDirect) {
                    x.fetch(0, st, p.K);
                    x.put(0, lds + buffer * S::kBuffer);
                }
                if constexpr (W::kDirect) {
                    v.fetch(0, st, p.K);
                    v.put(0, lds + buffer * S::kBuffer + X::kBytes);
                }
            }
        };
        constexpr int kFetches = X::kFetches + W::kFetches;
        // Large tiles: half of the wavefronts split their values in front of the products and the others behind them, so that
        // a SIMD's two use the vector and the matrix unit at the same time (4096 x 4096 x 4096 float32 596 instead of 610-639
        // us, w alone float32 327 instead of 335). In shorter steps the values are not there that early (1024 x 1024 x 1024
        // float32 23.8 instead of 22.0), and x alone is no gain (341 and 338).
        constexpr bool kApart = WF32 && RT * NT >= 16;
        const bool early = w >= S::kWaves / 2;
        auto step = [&](int st, auto odd) {
            constexpr int kSet = decltype(odd)::value;        // (st - st0) % 2: its buffer, and the registers of st + 2
            // what goes straight to LDS was asked for in front of the fetch of st + 2
            if (kLoads > 0) {
                if (st + 2 < st1 && st + 2 < full)
                    wait_loads<kFetches>();
                else
                    wait_loads<0>();
            }
            __syncthreads();                                  // step st is in LDS, and nobody reads the one before
            auto next = [&] {
                put(kSet ^ 1, kSet ^ 1);                      // behind the last step: something old, which nobody reads
                if (st + 3 < st1)
                    fetch(kSet ^ 1, st + 3);
            };
            if constexpr (kApart) {
                if (early)
                    put(kSet ^ 1, kSet ^ 1);
                if (st + 1 < st1)
                    load_or_put(st + 1, kSet ^ 1);
                if (early && st + 3 < st1)
                    fetch(kSet ^ 1, st + 3);
                compute(kSet, 0);
                if constexpr (S::kBK > 32)
                    compute(kSet, 1);
                if (!early)
                    next();
            } else {
                if (st + 1 < st1)
                    load_or_put(st + 1, kSet ^ 1);
                compute(kSet, 0);
                next();
                if constexpr (S::kBK > 32)
                    compute(kSet, 1);
            }
        };
        load_or_put(st0, 0);
        fetch(0, st0);
        put(0, 0);
        if (st0 + 1 < st1)
            fetch(1, st0 + 1);
        if (st0 + 2 < st1)
            fetch(0, st0 + 2);
        for (int st = st0; st < st1; st += 2) {
            step(st, std::integral_constant<int, 0>{});
            if (st + 1 < st1)
                step(st + 1, std::integral_constant<int, 1>{});
        }
    }
    __syncthreads();

    // A lane holds outputs 4 g .. 4 g + 3 of row col: through LDS, some strips of 16 rows at a time, so that a lane has 8
    // neighbouring outputs and a row's leave together.
    float* const mine = reinterpret_cast<float*>(lds) + w * (S::kStrips * 16 * S::kOutRow);
    constexpr int kCols = 16 * NT, kRowsAtOnce = kWave * 8 / kCols;
    const int i8 = lane / (kCols / 8), c8 = lane % (kCols / 8) * 8, n8 = n0 + wn * kCols + c8;
    const int have = p.N - n8;                                // outputs of this lane: 8, or a row's last, or none
    float bias[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        bias[i] = p.bias && i < have ? value_at(p.bias_bf16, p.bias, (size_t)n8 + i) : 0.0f;
    const bool partial = plan.splits > 1, add = p.residual && !partial;
    const size_t b0 = m0 + (size_t)(wr * RT) * 16;            // this wavefront's first row
    const int rows = b0 >= (size_t)p.B ? 0 : (size_t)p.B - b0 < (size_t)RT * 16 ? (int)((size_t)p.B - b0) : RT * 16;
    const int live = have > 0 ? rows : 0;
    const size_t at0 = b0 * (size_t)p.N + (size_t)n8;
    // Values of the residual come two turns ahead.
    constexpr int kTurnsAhead = 2;
    Raw queue[kTurnsAhead];
    auto ask = [&](int i, Raw& r) {
        if (add && i < live)
            r = have >= 8 ? load_raw<true>(p.residual_bf16, p.residual, at0 + (size_t)i * (size_t)p.N)
                          : load_short(p.residual_bf16, p.residual, at0 + (size_t)i * (size_t)p.N, have);
    };
#pragma unroll
    for (int q = 0; q < kTurnsAhead; ++q)
        ask(i8 + q * kRowsAtOnce, queue[q]);
#pragma unroll
    for (int part = 0; part < RT / S::kStrips; ++part) {
#pragma unroll
        for (int r = 0; r < S::kStrips; ++r)
#pragma unroll
            for (int f = 0; f < NT; ++f)
                *reinterpret_cast<f32x4*>(mine + (r * 16 + col) * S::kOutRow + f * 16 + 4 * g) = acc[part * S::kStrips + r][f];
        wave_lds_fence();
#pragma unroll 1
        for (int at_lds = i8; at_lds < S::kStrips * 16; at_lds += kRowsAtOnce) {
            const int i = part * S::kStrips * 16 + at_lds;
            const Raw residual = queue[0];
#pragma unroll
            for (int q = 0; q + 1 < kTurnsAhead; ++q)
                queue[q] = queue[q + 1];
            ask(i + kTurnsAhead * kRowsAtOnce, queue[kTurnsAhead - 1]);
            if (i >= live)
                continue;
            const f32x4 lo = *reinterpret_cast<const f32x4*>(mine + at_lds * S::kOutRow + c8);
            const f32x4 hi = *reinterpret_cast<const f32x4*>(mine + at_lds * S::kOutRow + c8 + 4);
            float o[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
            const size_t at = at0 + (size_t)i * (size_t)p.N;
            if (partial) {
                store_any<false>(plan.partial + (size_t)split * (size_t)p.B * (size_t)p.N, at, have, o);
                continue;
            }
            float more[8] = {};
            if (add)
                raw_values(p.residual_bf16, residual, more);
            linear_finish(p, bias, more, o);
            store_some(p.out_bf16, p.out, at, have, o);
        }
        wave_lds_fence();
    }
}

// A tile that a pair of types has, and what a step of it takes in us, as measured where all 256 CUs have one (or two) of
// them: products of 1024 to 8192 rows and K = 4096, less 4 us for the beginning and the end. The large tiles with a float32
// operand are 3 to 6 % faster than their number here, which is from before their wavefronts took turns (today's would be
// 2.25 of float32, 2.37 and 2.47 of one float32 side), and not every size gets its best tile: float32 1400 x 1024 -> 1024 has
// 35.3 us and could have 33.0, bfloat16 700 x 4096 -> 4096 51.6 and 46.5, 2048 x 2048 -> 1024 with float32 w 40.1 and 37.8.
struct TileCost {
    int rows, outputs, k;   // of x, of w, of a step
    float alone, paired;    // with one workgroup a CU, and with two (0: there is no room for two)
};

template <bool XF32, bool WF32, bool DIRECT, int RT, int NT, int WR, int WN, int RING, int BK>
hipError_t launch_linear_shape(const LinearArgs& p, const LinearPlan& plan, hipStream_t s)
{
    using S = LinearShape<XF32, WF32, DIRECT, RT, NT, WR, WN, RING, BK>;
    static_assert(16 * NT <= kWave, "a wavefront stores whole rows of its outputs");
    const void* f = reinterpret_cast<const void*>(&moe_linear_tiled_kernel<XF32, WF32, DIRECT, RT, NT, WR, WN, RING, BK>);
    if (S::kLds > 49152)
        if (hipError_t e = set_max_dynamic_lds(f, S::kLds))
            return e;
    const unsigned grid = (unsigned)((long long)plan.n_blocks * plan.m_blocks * plan.splits);
    hipLaunchKernelGGL((moe_linear_tiled_kernel<XF32, WF32, DIRECT, RT, NT, WR, WN, RING, BK>), dim3(grid), dim3(S::kThreads), S::kLds, s, p,
                       plan);
    return hipGetLastError();
}

// RING: buffers of a step, or kDeep; BK: values of k in a step.
template <bool XF32, bool WF32, int RT, int NT, int WR, int WN, int RING, int BK = 64>
hipError_t launch_linear_tile(const LinearArgs& p, const LinearPlan& plan, hipStream_t s)
{
    if ((XF32 && WF32) || p.K % 2 == 0)
        return launch_linear_shape<XF32, WF32, true, RT, NT, WR, WN, RING, BK>(p, plan, s);
    if constexpr (!(XF32 && WF32))
        return launch_linear_shape<XF32, WF32, false, RT, NT, WR, WN, 2, BK>(p, plan, s);
}

// One source file per pair of types. cost: of tile number i, false behind the last.
bool linear_cost_bf16(int tile, TileCost* cost);
bool linear_cost_mixed_w(int tile, TileCost* cost);           // bfloat16 x, float32 w
bool linear_cost_mixed_x(int tile, TileCost* cost);           // float32 x, bfloat16 w
bool linear_cost_f32(int tile, TileCost* cost);
hipError_t launch_linear_bf16(int tile, const LinearArgs& p, const LinearPlan& plan, hipStream_t s);
hipError_t launch_linear_mixed_w(int tile, const LinearArgs& p, const LinearPlan& plan, hipStream_t s);
hipError_t launch_linear_mixed_x(int tile, const LinearArgs& p, const LinearPlan& plan, hipStream_t s);
hipError_t launch_linear_f32(int tile, const LinearArgs& p, const LinearPlan& plan, hipStream_t s);

}  // namespace moed
