// The kernel of the dense product where one side has few rows: a decode batch times many weight rows, or many rows of x
// times few weight rows (a router of a few experts, a gate). Included by one source file per pair of types.
//
// A workgroup owns 16 rows of the side with many and 16 RT of the side with few. Its wavefronts share k: step st of kBK
// values is wavefront st % (all wavefronts of the tile)'s, so that together they stream through the rows. Each has a
// ring of LDS of its own that its loads fill and its fragments are read from: no barrier before the sums are added, in
// the order of the wavefronts, and the epilogue.
//
// Bound by the way of the rows from memory, and for short products by one round trip of it, the sum and the launch (us a
// call in a graph, eight sets of inputs in turn):
//                                          here    the tiles' kernel
//   32 x 4096 -> 4096 bfloat16             10.1      12.9
//   16 x 2048 -> 512 bfloat16               3.8       7.8
//   64 x 7168 -> 256, w float32             8.8      12.6             (both with k split and a second launch)
//   8192 x 4096 -> 16 bfloat16             18.6      19.2
// There a barrier a step lets the wavefronts wait together; here others' loads fill in for one's wait. Two sets of inputs
// stay in the Infinity Cache: 8.9 us for the first of these (3.9 TB/s) and 14.0 for the last (4.8); from HBM, with sixteen,
// 11.4-12.6 and 18.4 (2.7-3.0 and 3.7).
#pragma once

#include <type_traits>

#include "linear_common.h"

namespace moed {

// splits > 1: several workgroups share a tile's k; their sums go to partial [splits][B][N] instead of the epilogue.
struct SkinnyPlan {
    float* partial;
    int many_blocks, few_blocks, splits;
};

namespace {

constexpr int kSkinnyWaves = 8;

// FEW32, MANY32: that side is float32.
template <bool FEW32, bool MANY32, int RT>
struct SkinnyShape {
    static constexpr int kBK = FEW32 && MANY32 ? 32 : 64;
    static constexpr int kFU = kBK * (FEW32 ? 4 : 2) / 16, kMU = kBK * (MANY32 ? 4 : 2) / 16;  // units of a row and step
    static constexpr int kFewBytes = 16 * RT * kFU * 16, kManyBytes = 16 * kMU * 16;
    static constexpr int kFewLoads = kFewBytes / 1024, kManyLoads = kManyBytes / 1024, kLoads = kFewLoads + kManyLoads;
    static constexpr int kSlot = kFewBytes + kManyBytes;                  // of one wavefront
    static constexpr int kRing = 163840 / (kSkinnyWaves * kSlot) < 4 ? 163840 / (kSkinnyWaves * kSlot) : 4;
    static constexpr int kLds = kRing * kSkinnyWaves * kSlot;
    static_assert(kRing >= 2 && 16 * 16 * RT * 4 <= kRing * kSlot, "two steps, and room for the sums");
};

}  // namespace

// SWAPPED: the side with few rows is w, that with many x. DIRECT: rows begin at dwords (no bfloat16 rows of odd K), so that
// whole steps go straight to LDS.
template <bool FEW32, bool MANY32, bool SWAPPED, bool DIRECT, int RT>
__global__ void __launch_bounds__(kSkinnyWaves * kWave)
moe_linear_skinny_kernel(LinearArgs p, SkinnyPlan plan)
{
    using S = SkinnyShape<FEW32, MANY32, RT>;
    extern __shared__ __align__(16) uint8_t lds[];
    const int tid = threadIdx.x, lane = tid % kWave;
    const int w = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int g = lane / 16, col = lane % 16;
    const uint32_t lds0 = (uint32_t)(size_t)(__attribute__((address_space(3))) uint8_t*)lds;
    const uint8_t* const mine = lds + w * (S::kRing * S::kSlot);

    // the few blocks of one tile of many are neighbours on one XCD, so that its rows come from memory once
    const int item = xcd_contiguous(blockIdx.x, gridDim.x);
    const int fb = item % plan.few_blocks, rest = item / plan.few_blocks;
    const int split = rest / plan.many_blocks, mb = rest - split * plan.many_blocks;
    const int few0 = fb * 16 * RT;
    const size_t many0 = (size_t)mb * 16;
    const int few = SWAPPED ? p.N : p.B, many = SWAPPED ? p.B : p.N;      // rows
    const uint8_t* const fbase = static_cast<const uint8_t*>(SWAPPED ? p.w : p.x);
    const uint8_t* const mbase = static_cast<const uint8_t*>(SWAPPED ? p.x : p.w) + many0 * ((size_t)p.K * (MANY32 ? 4 : 2));
    const int flast = few - few0 < 16 * RT ? few - few0 - 1 : 16 * RT - 1;
    const int mlast = (size_t)many - many0 < 16 ? (int)((size_t)many - many0) - 1 : 15;

    // this lane's row and unit of each load
    uint32_t foff[S::kFewLoads], moff[S::kManyLoads];
    int funit[S::kFewLoads], munit[S::kManyLoads];
#pragma unroll
    for (int i = 0; i < S::kFewLoads; ++i) {
        const int r = i * (kWave / S::kFU) + lane / S::kFU;
        foff[i] = (uint32_t)(few0 + (r < flast ? r : flast)) * (uint32_t)((size_t)p.K * (FEW32 ? 4 : 2));
        funit[i] = (lane % S::kFU) ^ linear_swizzle<S::kFU, FEW32>(r);
    }
#pragma unroll
    for (int i = 0; i < S::kManyLoads; ++i) {
        const int r = i * (kWave / S::kMU) + lane / S::kMU;
        moff[i] = (uint32_t)(r < mlast ? r : mlast) * (uint32_t)((size_t)p.K * (MANY32 ? 4 : 2));
        munit[i] = (lane % S::kMU) ^ linear_swizzle<S::kMU, MANY32>(r);
    }
    const int full = DIRECT ? p.K / S::kBK : 0;
    // steps that end behind K, and rows that begin between dwords, go through registers
    u32x4 held_f[S::kFewLoads], held_m[S::kManyLoads];
    auto fetch = [&](int st) {
#pragma unroll
        for (int i = 0; i < S::kManyLoads; ++i)
            held_m[i] = row_unit<MANY32>(mbase + moff[i], st * S::kBK + munit[i] * (S::kBK / S::kMU), p.K);
#pragma unroll
        for (int i = 0; i < S::kFewLoads; ++i)
            held_f[i] = row_unit<FEW32>(fbase + foff[i], st * S::kBK + funit[i] * (S::kBK / S::kFU), p.K);
    };
    auto put = [&](int slot) {
        u32x4* const to = reinterpret_cast<u32x4*>(lds + w * (S::kRing * S::kSlot) + slot * S::kSlot) + lane;
#pragma unroll
        for (int i = 0; i < S::kManyLoads; ++i)
            to[S::kFewBytes / 16 + i * kWave] = held_m[i];
#pragma unroll
        for (int i = 0; i < S::kFewLoads; ++i)
            to[i * kWave] = held_f[i];
    };
    auto stage = [&](int st, int slot) {
        const int to = w * (S::kRing * S::kSlot) + slot * S::kSlot;
        if (st < full) {
            const uint8_t* fs = fbase + (size_t)st * (S::kFU * 16);
            const uint8_t* ms = mbase + (size_t)st * (S::kMU * 16);
#pragma unroll
            for (int i = 0; i < S::kManyLoads; ++i)
                load_to_lds16(ms, moff[i] + 16u * munit[i], lds0 + (uint32_t)(to + S::kFewBytes + i * 1024));
#pragma unroll
            for (int i = 0; i < S::kFewLoads; ++i)
                load_to_lds16(fs, foff[i] + 16u * funit[i], lds0 + (uint32_t)(to + i * 1024));
        } else {
            fetch(st);
            put(slot);
        }
    };

    f32x4 acc[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
        acc[r] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    auto compute = [&](int slot) {
        const uint8_t* fs = mine + slot * S::kSlot;
        const uint8_t* ms = fs + S::kFewBytes;
#pragma unroll
        for (int s = 0; s < S::kBK / 32; ++s) {
            bf16x8 mv[MANY32 ? 3 : 1];
            linear_fragment<MANY32, S::kMU>(ms, s, g, col, mv);
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                bf16x8 fv[FEW32 ? 3 : 1];
                linear_fragment<FEW32, S::kFU>(fs + r * 16 * S::kFU * 16, s, g, col, fv);
                linear_products<FEW32, MANY32>(mv, fv, acc[r]);
            }
        }
    };
    const int all = (p.K + S::kBK - 1) / S::kBK, stride = plan.splits * kSkinnyWaves;
    const int st0 = split * kSkinnyWaves + w;
    const int count = st0 < all ? (all - st0 + stride - 1) / stride : 0;  // this wavefront's steps
    constexpr int kAhead = S::kRing - 1;
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        if (i < count)
            stage(st0 + i * stride, i);
    int slot = 0;
    for (int i = 0; i < count; ++i) {
        const int free = slot == 0 ? kAhead : slot - 1;
        const bool more = i + kAhead < count;
        const int later = st0 + (i + kAhead) * stride;
        if constexpr (DIRECT) {
            if (more) {
                wait_lds();                                   // the fragments of the step before, whose place is taken now
                stage(later, free);
                wait_loads<kAhead * S::kLoads>();             // all but the loads of the steps behind this one
            } else {
                wait_loads<0>();
            }
            wave_lds_fence();
            compute(slot);
        } else {
            if (more)
                fetch(later);                                 // comes while this step is multiplied
            wave_lds_fence();
            compute(slot);
            if (more)
                put(free);
        }
        slot = slot + 1 == S::kRing ? 0 : slot + 1;
    }
    // Sums of the wavefronts: [wavefront][few][many]. Their 16-byte writes are all of the kernel's LDS bank conflicts, 24
    // cycles a fragment whatever K (18 % of its LDS cycles at 32 x 4096 -> 4096, 6 % at K = 16384).
    float* const sums = reinterpret_cast<float*>(lds + w * (S::kRing * S::kSlot));
    wave_lds_fence();
#pragma unroll
    for (int r = 0; r < RT; ++r)
        *reinterpret_cast<f32x4*>(sums + (r * 16 + col) * 16 + 4 * g) = acc[r];
    __syncthreads();
    if (tid >= 256 * RT)
        return;
    const int f = SWAPPED ? tid % (16 * RT) : tid / 16, m = SWAPPED ? tid / (16 * RT) : tid % 16;
    float v = 0.0f;
#pragma unroll
    for (int q = 0; q < kSkinnyWaves; ++q)
        v += *reinterpret_cast<const float*>(lds + q * (S::kRing * S::kSlot) + (f * 16 + m) * 4);
    if (f > flast || m > mlast)
        return;
    const size_t b = SWAPPED ? many0 + m : (size_t)(few0 + f);
    const int n = SWAPPED ? few0 + f : (int)many0 + m;
    if (plan.splits > 1)
        plan.partial[((size_t)split * (size_t)p.B + b) * (size_t)p.N + n] = v;
    else
        linear_store(p, v, b, n);
}

template <bool FEW32, bool MANY32, bool SWAPPED, bool DIRECT, int RT>
hipError_t launch_skinny_shape(const LinearArgs& p, const SkinnyPlan& plan, hipStream_t s)
{
    using S = SkinnyShape<FEW32, MANY32, RT>;
    static_assert(256 * RT <= kSkinnyWaves * kWave, "a thread for each output");
    const void* f = reinterpret_cast<const void*>(&moe_linear_skinny_kernel<FEW32, MANY32, SWAPPED, DIRECT, RT>);
    if (S::kLds > 49152)
        if (hipError_t e = set_max_dynamic_lds(f, S::kLds))
            return e;
    const unsigned grid = (unsigned)((long long)plan.many_blocks * plan.few_blocks * plan.splits);
    hipLaunchKernelGGL((moe_linear_skinny_kernel<FEW32, MANY32, SWAPPED, DIRECT, RT>), dim3(grid), dim3(kSkinnyWaves * kWave),
                       S::kLds, s, p, plan);
    return hipGetLastError();
}

// rt: 16-row fragments of the side with few, 1 or 2.
template <bool X32, bool W32>
hipError_t launch_skinny(bool swapped, int rt, const LinearArgs& p, const SkinnyPlan& plan, hipStream_t s)
{
    const bool direct = (X32 && W32) || p.K % 2 == 0;
#define MOED_SK(F, M, SW) \
    (direct ? (rt == 1 ? launch_skinny_shape<F, M, SW, true, 1>(p, plan, s) : launch_skinny_shape<F, M, SW, true, 2>(p, plan, s)) \
            : (rt == 1 ? launch_skinny_shape<F, M, SW, (F && M), 1>(p, plan, s) : launch_skinny_shape<F, M, SW, (F && M), 2>(p, plan, s)))
    return swapped ? MOED_SK(W32, X32, true) : MOED_SK(X32, W32, false);
#undef MOED_SK
}

// One source file per pair of types.
hipError_t launch_skinny_bf16(bool swapped, int rt, const LinearArgs& p, const SkinnyPlan& plan, hipStream_t s);
hipError_t launch_skinny_mixed_w(bool swapped, int rt, const LinearArgs& p, const SkinnyPlan& plan, hipStream_t s);
hipError_t launch_skinny_mixed_x(bool swapped, int rt, const LinearArgs& p, const SkinnyPlan& plan, hipStream_t s);
hipError_t launch_skinny_f32(bool swapped, int rt, const LinearArgs& p, const SkinnyPlan& plan, hipStream_t s);

}  // namespace moed
