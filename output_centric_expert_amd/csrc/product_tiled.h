// The kernel of the products grouped by expert: tiles of rows x weight rows through LDS, matrix instructions on what
// it holds. Included by one source file per kind of rows.
//
// A workgroup walks tiles (expert, rows, block of outputs) with a stride of the grid. A step is 128 values of K: its
// weight rows, rows and block scales go from memory straight to LDS, two buffers of each; while a tile is stored, the
// next one's first step is on its way. The mathematics is in product_common.h; what bounds a call:
//  - up to about 50 rows an expert, the weights' bytes: 512 tokens of 8 of 128 experts, K = 2048, N = 768, gate and up
//    in MXFP8 take 83 us with bfloat16 rows (5.1 TB/s of codes and scales), 90 with MXFP8 rows decoded to it, 80 with
//    MXFP8 rows on the scaled instructions;
//  - beyond, the matrix instructions and what goes with them. On the scaled ones 8192 tokens take 280-288 us (1.43-1.47
//    PFLOP/s; the same loop without loads 224 us: the clock falls to 1.7 GHz under these instructions), of which the
//    tiles' beginnings and ends are a sixth. With bfloat16 rows (461-491 us) the decode of the weights (16 conversions
//    for 4 * RT matrix instructions) comes on top, with MXFP8 rows decoded to it (522-540 us) also the rows' (16 for
//    4 * NT, by every wavefront that reads them).
// What did not pay: fragments of the weights read straight from memory (a load of 16 rows x 64 bytes runs at a quarter
// of the rate of one of 8 rows x 128 bytes); two groups of wavefronts taking turns between LDS and the matrix unit, and
// loads spread among the matrix instructions (both wait longer for the loads than they save).
#pragma once

#include <type_traits>

#include "product_common.h"

namespace moed {

// How rows enter the matrix instructions.
constexpr int kRowsBF16 = 0;      // bfloat16 rows, weights decoded to bfloat16
constexpr int kRowsMX = 1;        // MXFP8 rows and MX weights as stored, scaled matrix instructions
constexpr int kRowsMXExact = 2;   // MXFP8 rows and weights both decoded to bfloat16

// Block scales that the decode to bfloat16 holds exactly with any code (255 is NaN either way).
template <bool FP4>
__device__ __forceinline__ bool exact_scale(uint32_t c)
{
    constexpr uint32_t lo = FP4 ? kExactScaleLoFP4 : kExactScaleLoFP8, hi = FP4 ? kExactScaleHiFP4 : kExactScaleHiFP8;
    return c - lo <= hi - lo || c == 255u;
}

static __device__ const u32x4 kZeros = {0, 0, 0, 0};   // source of the values behind the end of a row

// 16 bytes per lane from global memory straight to LDS: lane i of the wavefront
// writes base + 16 i (base uniform). No register receives the data; the caller
// waits on vmcnt before a barrier. Written as asm because the compiler makes
// every later LDS read wait for the builtin's load, whatever buffer it fills.
// The address is a uniform base plus a lane's 32-bit offset.
__device__ __forceinline__ void load_to_lds16(const uint8_t* from, uint32_t offset, uint32_t base)
{
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(offset), "s"(from), "s"(base)
                 : "memory", "m0");
}

// The same from an address of each lane's own.
__device__ __forceinline__ void load_to_lds16(const uint8_t* from, uint32_t base)
{
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(from), "s"(base) : "memory", "m0");
}

__device__ __forceinline__ void load_to_lds4(const void* from, uint32_t base)
{
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off" ::"v"(from), "s"(base) : "memory", "m0");
}

template <int ROWS, bool FP4, int OUT, int RT, int NT, int WR, int WN>
struct Shape {
    static constexpr bool kMX = ROWS == kRowsMX;
    static constexpr int kWaves = WR * WN, kThreads = kWaves * kWave;
    static constexpr int kBM = 16 * RT * WR;                  // rows of a tile
    static constexpr int kBN = 16 * NT * WN;                  // weight rows of a tile
    static constexpr int kBK = 128;                           // values of a step
    static constexpr int kRU = ROWS == kRowsBF16 ? 16 : 8;    // 16-byte units of a row and step
    static constexpr int kWU = FP4 ? 4 : 8;                   // ... of a weight row and step
    static constexpr int kRowLoads = (kBM * kRU + kThreads - 1) / kThreads;
    static constexpr int kWLoads = (kBN * kWU + kThreads - 1) / kThreads;
    static constexpr int kRowBytes = kBM * kRU * 16, kWBytes = kBN * kWU * 16;
    static constexpr int kWAt = 2 * kRowBytes;
    // block scales: of every weight row, and of every row in MXFP8
    static constexpr int kScaleRows = (kBN + (ROWS != kRowsBF16 ? kBM : 0) + kWave - 1) / kWave * kWave;
    static constexpr int kScaleLoads = (kScaleRows + kThreads - 1) / kThreads;
    static constexpr int kScaleBytes = kScaleRows * 16;
    // 16 rows of a wavefront's outputs on their way out
    static constexpr int kOutBytes = OUT == kOutBF16 ? 2 : OUT == kOutF32 ? 4 : 1;
    static constexpr int kScaleAt = kWAt + 2 * kWBytes;
    static constexpr int kEnd = kScaleAt + 2 * kScaleBytes;
    static constexpr int scratch_row(int out_frags) { return OUT == kOutF32 ? 0 : out_frags * 16 * kOutBytes + 16; }
    // it lies in the second row buffer, which is free between a tile's last and the next one's second step
    static constexpr bool inside(int out_frags) { return kWaves * 16 * scratch_row(out_frags) <= kRowBytes; }
    static constexpr int scratch_at(int out_frags) { return inside(out_frags) ? kRowBytes : kEnd; }
    static constexpr int bad_at(int out_frags) { return kEnd + (inside(out_frags) ? 0 : kWaves * 16 * scratch_row(out_frags)); }
    static constexpr int slots_at(int out_frags) { return bad_at(out_frags) + 2 * kBM; }
    static constexpr int kSlots = (kBM + kWave - 1) / kWave * kWave;
    static constexpr int lds(int out_frags) { return slots_at(out_frags) + 4 * kSlots; }
    static_assert(kBM * kRU % kWave == 0 && kBN * kWU % kWave == 0, "whole loads per wavefront");
    static_assert((kThreads / kRU) % 8 == 0 && (kThreads / kWU) % 8 == 0, "a thread's loads share their place in the row");
    // loads of a step's weights by the wavefront that has the fewest
    static constexpr int kWeightLoads = kBN * kWU / kThreads;
};

template <int N>
__device__ __forceinline__ void wait_loads()
{
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Units of a row are stored at c ^ swizzle(row), so that the lanes that read one
// unit of 8 neighbouring rows together meet different banks.
template <int UNITS>
__device__ __forceinline__ int swizzle(int row)
{
    return UNITS >= 8 ? row & 7 : (row >> 1) & 3;
}

// Byte offset of unit c of row `col` (below 16) of a fragment; the same unit of
// fragment f lies f * 16 * UNITS * 16 bytes on.
template <int UNITS>
__device__ __forceinline__ int unit_at(int col, int c)
{
    return (col * UNITS + (c ^ swizzle<UNITS>(col))) * 16;
}

__device__ __forceinline__ u32x4 lds16(const uint8_t* p) { return *reinterpret_cast<const u32x4*>(p); }

// f(N) with the smallest of RT, RT/2, RT/4 .. (as a constant) that is at least
// `live`: a tile's last rows take no more matrix instructions than they need.
template <int RT, typename F>
__device__ __forceinline__ void row_parts(int live, F&& f)
{
    if constexpr (RT >= 4) {
        if (live <= RT / 2) {
            row_parts<RT / 2>(live, f);
            return;
        }
    }
    f(std::integral_constant<int, RT>{});
}

// One tile: rows m0 .. of expert e, outputs n0 .. .
struct Tile {
    int e, m0, n0, rows, row0;
    bool live;
};

template <int ROWS, bool FP4, bool GLU, int OUT, int RT, int NT, int WR, int WN>
__global__ void __launch_bounds__(WR * WN * kWave)
moe_product_tiled_kernel(ProductArgs p, int nblk, int group_blocks, int contiguous)
{
    using S = Shape<ROWS, FP4, OUT, RT, NT, WR, WN>;
    constexpr int kOutFrags = GLU ? NT / 2 : NT;
    constexpr int kNeurons = 16 * kOutFrags * WN;             // outputs of a tile
    constexpr int kScratchRow = S::scratch_row(kOutFrags);
    constexpr int kAhead = 1;
    // rounded outputs of rows and weights decoded to bfloat16: a tile that meets a block scale which the decode does not
    // hold exactly is computed once more, with the scaled instructions
    constexpr bool kRedo = ROWS == kRowsMXExact && OUT != kOutF32;
    extern __shared__ __align__(16) uint8_t lds[];
    uint8_t* const bad = lds + S::bad_at(kOutFrags);          // [2][kBM]: rows without a source
    int* const first = reinterpret_cast<int*>(lds + S::lds(kOutFrags));           // tiles before each expert
    int* const begin = first + p.E + 1;                       // its first row
    __shared__ int wsum[S::kWaves];
    __shared__ int redo[2];                                   // by the tile's parity
    const int tid = threadIdx.x, lane = tid % kWave;
    const int w = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int g = lane / 16, col = lane % 16;
    const int wr = w / WN, wn = w % WN;
    const int tiles = build_tiles<S::kThreads>(first, begin, p.offsets, p.E, p.R, S::kBM, wsum);
    const int items = tiles * nblk;                           // below 2^31: checked by the host
    const size_t w_row = FP4 ? (size_t)p.K / 2 : (size_t)p.K, s_row = (size_t)p.s_row;
    const size_t a_row = ROWS == kRowsBF16 ? 2 * (size_t)p.K : (size_t)p.K;
    const uint32_t lds0 = (uint32_t)(size_t)(__attribute__((address_space(3))) uint8_t*)lds;

    // items of one expert are neighbours; within it blocks of weight rows in
    // groups, so that a group's weights and the expert's rows meet in one L2
    auto find = [&](int item) {
        Tile t;
        t.live = false;
        t.e = t.m0 = t.n0 = t.rows = t.row0 = 0;
        if (item < 0 || item >= items)                        // negative: past 2^31
            return t;
        const int e = tile_expert(first, p.E, item / nblk);
        if (e >= p.E)
            return t;
        const int mt = first[e + 1] - first[e];
        const int local = item - first[e] * nblk;
        const int grp = local / (group_blocks * mt);
        const int rest = local - grp * group_blocks * mt;
        const int in_grp = nblk - grp * group_blocks < group_blocks ? nblk - grp * group_blocks : group_blocks;
        t.e = __builtin_amdgcn_readfirstlane(e);
        t.n0 = __builtin_amdgcn_readfirstlane((grp * group_blocks + rest % in_grp) * kNeurons);
        t.m0 = __builtin_amdgcn_readfirstlane((rest / in_grp) * S::kBM);
        t.row0 = __builtin_amdgcn_readfirstlane(begin[t.e]);
        t.rows = __builtin_amdgcn_readfirstlane(begin[t.e + 1]) - t.row0;
        t.live = t.m0 < t.rows && t.n0 < p.N;
        return t;
    };
    const int rc = (tid % S::kRU) ^ swizzle<S::kRU>(tid / S::kRU);        // this thread's unit within a row and step
    const int wc = (tid % S::kWU) ^ swizzle<S::kWU>(tid / S::kWU);
    auto tile_row = [&](const Tile& t, int r) {                           // rows behind the last repeat it
        return t.row0 + (t.m0 + r < t.rows ? t.m0 + r : t.rows - 1);
    };
    // slots of a tile's rows, fetched to LDS while the tile before it is computed
    const int* const slots = reinterpret_cast<const int*>(lds + S::slots_at(kOutFrags));
    auto fetch_slots = [&](const Tile& t) {
        if (p.order)
#pragma unroll
            for (int i = 0; i < (S::kSlots + S::kThreads - 1) / S::kThreads; ++i)
                if (i * S::kThreads + w * kWave < S::kSlots)
                    load_to_lds4(p.order + tile_row(t, i * S::kThreads + tid),
                                 lds0 + S::slots_at(kOutFrags) + (uint32_t)(i * S::kThreads + w * kWave) * 4u);
    };
    // row of `a` that row r of the tile reads, -1 for none
    auto source = [&](const Tile& t, int r) {
        return p.order ? source_row(p, slots[r]) : tile_row(t, r);
    };

    // Sources: uniform bases and 32-bit offsets (a wavefront's load of weights
    // lies within one fragment, so its matrix is uniform too); addresses for the
    // scales.
    const uint8_t *rbase = nullptr, *wbase = nullptr, *ubase = nullptr;
    uint32_t roff[S::kRowLoads], woff[S::kWLoads];            // woff: uniform, in rows
    const uint8_t* ssrc[S::kScaleLoads];
    const uint32_t wlane = (uint32_t)(lane / S::kWU) * (uint32_t)w_row + 16u * wc;
    auto is_up = [&](int place) { return GLU && place / 16 % NT >= NT / 2; };       // place: weight row of the tile
    // Row of its expert's matrix; N is a multiple of 32, so the 16 rows of a fragment lie before or behind its end
    // together, and those behind repeat fragment 0 (they are not stored).
    auto weight_row = [&](const Tile& t, int place) {
        const int f = place / 16 % NT;
        const int n = t.n0 + (place / (16 * NT) * kOutFrags + (GLU && f >= NT / 2 ? f - NT / 2 : f)) * 16 + place % 16;
        return (uint32_t)(n < p.N ? n : place % 16);
    };
    auto point = [&](const Tile& t, int parity) {
        rbase = static_cast<const uint8_t*>(p.a) + (p.order ? 0 : (size_t)(t.row0 + t.m0) * a_row);
        const size_t m = (size_t)t.e * (size_t)p.N;
        wbase = p.w_q + m * w_row;
        if constexpr (GLU)
            ubase = p.u_q + m * w_row;
#pragma unroll
        for (int i = 0; i < S::kRowLoads; ++i) {
            const int r = i * (S::kThreads / S::kRU) + tid / S::kRU;
            const int from = source(t, r < S::kBM ? r : S::kBM - 1);
            roff[i] = (uint32_t)(from < 0 ? 0 : p.order ? from : from - (t.row0 + t.m0)) * (uint32_t)a_row + 16u * rc;
            if (tid % S::kRU == 0 && r < S::kBM)
                bad[parity * S::kBM + r] = from < 0;
        }
#pragma unroll
        for (int i = 0; i < S::kWLoads; ++i)                  // first of this wavefront's rows in load i
            woff[i] = weight_row(t, i * (S::kThreads / S::kWU) + w * (kWave / S::kWU));
#pragma unroll
        for (int i = 0; i < S::kScaleLoads; ++i) {
            const int place = i * S::kThreads + tid;
            if (ROWS != kRowsBF16 && place >= S::kBN) {
                const int from = source(t, place - S::kBN < S::kBM ? place - S::kBN : S::kBM - 1);
                ssrc[i] = p.a_s + (size_t)(from < 0 ? 0 : from) * s_row;
            } else {
                const int at = place < S::kBN ? place : 0;
                ssrc[i] = (is_up(at) ? p.u_s : p.w_s) + (m + weight_row(t, at)) * s_row;
            }
        }
    };
    const uint8_t* const zeros = reinterpret_cast<const uint8_t*>(&kZeros);
    const int full = p.K / S::kBK, steps = (p.K + S::kBK - 1) / S::kBK;
    auto stage_rows = [&](int st) {
        const uint32_t to = lds0 + (uint32_t)(st & 1) * S::kRowBytes + (uint32_t)w * 1024u;
        const uint8_t* from = rbase + (size_t)st * (S::kRU * 16);
        if (st < full) {
#pragma unroll
            for (int i = 0; i < S::kRowLoads; ++i)
                if (S::kBM * S::kRU % S::kThreads == 0 || i * S::kThreads + w * kWave < S::kBM * S::kRU)
                    load_to_lds16(from, roff[i], to + i * S::kThreads * 16);
        } else {                                              // a K that is no multiple of 128: zeros behind its end
            const bool in = st * S::kBK + rc * (S::kBK / S::kRU) < p.K;
#pragma unroll
            for (int i = 0; i < S::kRowLoads; ++i)
                if (S::kBM * S::kRU % S::kThreads == 0 || i * S::kThreads + w * kWave < S::kBM * S::kRU)
                    load_to_lds16(in ? from + roff[i] : zeros, to + i * S::kThreads * 16);
        }
    };
    auto stage_weights = [&](int st) {
        const uint32_t to = lds0 + S::kWAt + (uint32_t)(st & 1) * S::kWBytes + (uint32_t)w * 1024u;
        const bool in = st < full || st * S::kBK + wc * (S::kBK / S::kWU) < p.K;
#pragma unroll
        for (int i = 0; i < S::kWLoads; ++i) {
            if (S::kBN * S::kWU % S::kThreads != 0 && i * S::kThreads + w * kWave >= S::kBN * S::kWU)
                continue;                                     // whole wavefronts
            const uint8_t* from = (is_up(i * (S::kThreads / S::kWU) + w * (kWave / S::kWU)) ? ubase : wbase) +
                                  (size_t)woff[i] * w_row + (size_t)st * (S::kWU * 16);
            if (st < full)
                load_to_lds16(from, wlane, to + i * S::kThreads * 16);
            else
                load_to_lds16(in ? from + wlane : zeros, to + i * S::kThreads * 16);
        }
    };
    // Block scales are fetched 16 bytes (four steps) of a row at a time: a load
    // that takes four bytes of each of 64 rows costs the cache about as much as
    // one that takes a line of each. Where a row is no multiple of 16, the last
    // fetch is of the row's last 16 bytes, the wanted ones at its end.
    auto scales_from = [&](int chunk) { return 16 * chunk + 16 <= p.s_row ? 16 * chunk : p.s_row - 16; };
    auto stage_scales = [&](int chunk) {
        const uint32_t to = lds0 + S::kScaleAt + (uint32_t)(chunk & 1) * S::kScaleBytes;
        const int from = scales_from(chunk);
#pragma unroll
        for (int i = 0; i < S::kScaleLoads; ++i) {
            const int place = i * S::kThreads + w * kWave;    // of this wavefront's first lane
            if (S::kScaleRows % S::kThreads == 0 || place < S::kScaleRows)
                load_to_lds16(ssrc[i] + from, to + place * 16);
        }
    };
    // the steps a tile begins with
    auto stage_first = [&]() {
        stage_scales(0);
        stage_rows(0);
        stage_weights(0);
        if (steps > 1)
            stage_weights(1);
    };

    // this lane's places in the buffers
    const int w0 = wn * NT * 16 * S::kWU * 16, r0 = wr * RT * 16 * S::kRU * 16;
    constexpr int kWFrag = 16 * S::kWU * 16, kRFrag = 16 * S::kRU * 16;      // bytes of a fragment
    f32x4 acc[RT][NT];
    bool strange = false;                                     // this lane met such a scale (kRedo)
    // One step's products for the first n fragments of rows, with the scaled instructions or on bfloat16. `release` is
    // called once the step's weights and scales are in registers.
    auto compute = [&](int st, auto n, auto scaled, auto release) {
        constexpr int N = decltype(n)::value;
        const uint8_t* wb = lds + S::kWAt + (st & 1) * S::kWBytes + w0;
        const uint8_t* rb = lds + (st & 1) * S::kRowBytes + r0;
        const int chunk = st / 4;
        const uint8_t* sb = lds + S::kScaleAt + (chunk & 1) * S::kScaleBytes + (4 * st - scales_from(chunk)) + 16 * col + g;
        const uint8_t* wsb = sb + wn * NT * 256;
        const uint8_t* rsb = sb + (S::kBN + wr * RT * 16) * 16;
        if constexpr (decltype(scaled)::value) {
            i32x8 wv[NT], av[kAhead + 1];
            int wsc[NT], asc[RT];
            const uint8_t* rlo = rb + unit_at<8>(col, g);
            const uint8_t* rhi = rb + unit_at<8>(col, 4 + g);
            auto read_a = [&](int r) {
                const u32x4 lo = lds16(rlo + r * kRFrag), hi = lds16(rhi + r * kRFrag);
                av[r % (kAhead + 1)] =
                    i32x8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
            };
            auto read_w = [&](int f) {
                const u32x4 lo = lds16(wb + unit_at<S::kWU>(col, g) + f * kWFrag);
                const u32x4 hi = FP4 ? u32x4{0, 0, 0, 0} : lds16(wb + unit_at<S::kWU>(col, FP4 ? 0 : 4 + g) + f * kWFrag);
                wv[f] = i32x8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
                wsc[f] = wsb[f * 256];
            };
#pragma unroll
            for (int f = 0; f < NT; ++f)
                read_w(f);
#pragma unroll
            for (int r = 0; r < RT; ++r)
                asc[r] = rsb[r * 256];
#pragma unroll
            for (int r = 0; r < kAhead && r < N; ++r)
                read_a(r);
            release();
            __builtin_amdgcn_sched_barrier(0);
            // fragments of rows are read kAhead before their use, so that the reads of one pass under
            // the matrix instructions of the others
#pragma unroll
            for (int r = 0; r < N; ++r) {
                if (r + kAhead < N)
                    read_a(r + kAhead);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int f = 0; f < NT; ++f)
                    acc[r][f] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        wv[f], av[r % (kAhead + 1)], acc[r][f], FP4 ? 4 : 0, 0, 0, wsc[f], 0, asc[r]);
                __builtin_amdgcn_sched_barrier(0);
            }
        } else {
            // lane group g multiplies the block 32g .. 32g+31 of the step, 8 values per instruction
            u32x4 wq[NT][FP4 ? 1 : 2];
            float wsc[NT], asc[ROWS == kRowsMXExact ? RT : 1];
            bool outside = false;
#pragma unroll
            for (int f = 0; f < NT; ++f) {
                if constexpr (FP4) {
                    wq[f][0] = lds16(wb + unit_at<4>(col, g) + f * kWFrag);
                } else {
                    wq[f][0] = lds16(wb + unit_at<8>(col, 2 * g) + f * kWFrag);
                    wq[f][1] = lds16(wb + unit_at<8>(col, 2 * g + 1) + f * kWFrag);
                }
                const uint32_t c = wsb[f * 256];
                wsc[f] = ue8m0_to_f32(c);
                if constexpr (kRedo)
                    outside |= !exact_scale<FP4>(c);
            }
            if constexpr (ROWS == kRowsMXExact) {
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    const uint32_t c = rsb[r * 256];
                    asc[r] = ue8m0_to_f32(c);
                    if constexpr (kRedo)
                        outside |= r < N && !exact_scale<false>(c);
                }
            }
            release();
            if constexpr (kRedo) {
                if (__any(outside)) {                         // rare; blocks of zeros decode exactly whatever their scale
#pragma unroll
                    for (int f = 0; f < NT; ++f) {
                        uint32_t any = 0;
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            any |= FP4 ? wq[f][0][i] & 0x77777777u : (wq[f][0][i] | wq[f][FP4 ? 0 : 1][i]) & 0x7F7F7F7Fu;
                        strange |= any != 0 && !exact_scale<FP4>(wsb[f * 256]);
                    }
#pragma unroll
                    for (int r = 0; r < N; ++r) {
                        const u32x4 lo = lds16(rb + unit_at<8>(col, 2 * g) + r * kRFrag);
                        const u32x4 hi = lds16(rb + unit_at<8>(col, 2 * g + 1) + r * kRFrag);
                        uint32_t any = 0;
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            any |= (lo[i] | hi[i]) & 0x7F7F7F7Fu;
                        strange |= any != 0 && !exact_scale<false>(rsb[r * 256]);
                    }
                }
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                bf16x8 wv[NT];
#pragma unroll
                for (int f = 0; f < NT; ++f) {
                    if constexpr (FP4) {
                        wv[f] = decode8_scaled_fp4(wq[f][0][q], wsc[f]);
                    } else {
                        const u32x4 c = wq[f][q / 2];
                        wv[f] = decode8_scaled((q & 1) ? u32x2{c.z, c.w} : u32x2{c.x, c.y}, wsc[f]);
                    }
                }
#pragma unroll
                for (int r = 0; r < N; ++r) {
                    bf16x8 av;
                    if constexpr (ROWS == kRowsMXExact) {
                        const u32x4 c = lds16(rb + unit_at<8>(col, 2 * g + q / 2) + r * kRFrag);
                        av = decode8_scaled((q & 1) ? u32x2{c.z, c.w} : u32x2{c.x, c.y}, asc[r]);
                    } else {
                        av = __builtin_bit_cast(bf16x8, lds16(rb + unit_at<16>(col, 4 * g + q) + r * kRFrag));
                    }
#pragma unroll
                    for (int f = 0; f < NT; ++f)
                        acc[r][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv[f], av, acc[r][f], 0, 0, 0);
                }
            }
        }
    };

    int item = contiguous ? xcd_contiguous(blockIdx.x, gridDim.x) : (int)blockIdx.x;
    Tile t = find(item);
    int parity = 0;
    if (t.live)
        fetch_slots(t);
    wait_loads<0>();
    __syncthreads();
    if (t.live) {
        point(t, 0);
        stage_first();
    }
    while (item >= 0 && item < items) {
        Tile next = find(item + (int)gridDim.x);
        __syncthreads();                                      // everybody has this tile's slots
        if (next.live)
            fetch_slots(next);
        // all steps of the tile; the first ones are on their way
        auto run_steps = [&](auto scaled) {
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int f = 0; f < NT; ++f)
                    acc[r][f] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            if (!t.live)
                return;
            // row fragments of this wavefront that hold rows
            row_parts<RT>((t.rows - t.m0 - wr * RT * 16 + 15) / 16, [&](auto n) {
                for (int st = 0; st < steps; ++st) {
                    // A step's weights are asked for nearly two steps ahead (they come from far, and their buffer is
                    // free as soon as every wavefront has its fragments), its rows one step ahead. Step st is in LDS
                    // once this wavefront's loads of it, and then everybody's, are done.
                    if (st + 1 < steps)
                        wait_loads<S::kWeightLoads>();
                    else
                        wait_loads<0>();
                    __syncthreads();
                    if (st + 1 < steps)
                        stage_rows(st + 1);
                    compute(st, n, scaled, [&] {
                        __syncthreads();                          // everybody has the step's weights
                        if ((st & 3) == 2 && st + 2 < steps)
                            stage_scales(st / 4 + 1);
                        if (st + 2 < steps)
                            stage_weights(st + 2);
                    });
                }
            });
        };
        if constexpr (kRedo) {
            strange = false;
            if (tid == 0)
                redo[parity] = 0;                             // read last two tiles ago
        }
        run_steps(std::bool_constant<S::kMX>{});
        if constexpr (kRedo)
            if (__any(strange) && lane == 0)
                redo[parity] = 1;
        // the next tile's first steps are on their way while this one is stored
        wait_loads<0>();                                      // its slots, where this tile had no steps to wait in
        __syncthreads();
        if constexpr (kRedo) {
            if (redo[parity]) {                               // the same for all
                stage_first();
                run_steps(std::true_type{});
                wait_loads<0>();
                __syncthreads();
            }
        }
        if (next.live) {
            point(next, parity ^ 1);
            stage_first();
        }
        if (t.live) {
            uint8_t* mine = lds + S::scratch_at(kOutFrags) + w * 16 * kScratchRow;
            const int nw = t.n0 + wn * kOutFrags * 16;        // this wavefront's first output
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                if (t.m0 + (wr * RT + r) * 16 >= t.rows)
                    break;
                const bool none = bad[parity * S::kBM + (wr * RT + r) * 16 + col];
                f32x4 o[kOutFrags];
#pragma unroll
                for (int f = 0; f < kOutFrags; ++f)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float v = acc[r][f][i];
                        if constexpr (GLU)
                            v = swiglu(v, acc[r][f + NT / 2][i]);
                        o[f][i] = none ? __builtin_nanf("") : v;
                    }
                store_tile_rows<OUT, kOutFrags>(p, mine, kScratchRow, t.row0, t.m0 + (wr * RT + r) * 16, t.rows, nw, o);
            }
        }
        item += (int)gridDim.x;
        t = next;
        parity ^= 1;
    }
}

template <int ROWS, bool FP4, bool GLU, int OUT, int RT, int NT, int WR, int WN>
hipError_t launch_shape(const ProductArgs& p, int avg, hipStream_t s)
{
    using S = Shape<ROWS, FP4, OUT, RT, NT, WR, WN>;
    constexpr int kOutFrags = GLU ? NT / 2 : NT;
    constexpr int kNeurons = 16 * kOutFrags * WN;
    const size_t lds = S::lds(kOutFrags) + ((size_t)p.E + 1) * 8;
    const void* f = reinterpret_cast<const void*>(&moe_product_tiled_kernel<ROWS, FP4, GLU, OUT, RT, NT, WR, WN>);
    if (lds > 49152)
        if (hipError_t e = set_max_dynamic_lds(f, (int)lds))
            return e;
    const int nblk = (p.N + kNeurons - 1) / kNeurons;
    const long long tiles = (long long)p.R / S::kBM + (p.R < p.E ? p.R : p.E);
    const int per_cu = (int)((size_t)163840 / (lds + 64));
    long long grid = tiles * nblk;
    const long long most = 256LL * (per_cu < 1 ? 1 : per_cu > 4 ? 4 : per_cu);
    grid = grid < most ? grid : most;
    // weight rows of about 512 KiB per group of blocks (2 MiB: matmul of 8192 tokens, K = 768, N = 2048, 183 us
    // instead of 171; no difference where K is 2048)
    const long long bytes = (long long)S::kBN * p.K / (FP4 ? 2 : 1);
    long long group = (512LL << 10) / bytes;
    group = group < 1 ? 1 : group > nblk ? nblk : group;
    // Neighbouring tiles on one XCD where an expert has several tiles of rows, which then share its weights in one L2
    // (gate_up of 8192 tokens 298 instead of 321 us); otherwise in turn over the XCDs (8 tokens: 34 instead of 37 us).
    const bool contiguous = avg > S::kBM;
    hipLaunchKernelGGL((moe_product_tiled_kernel<ROWS, FP4, GLU, OUT, RT, NT, WR, WN>), dim3((unsigned)grid),
                       dim3(S::kThreads), lds, s, p, nblk, (int)group, contiguous ? 1 : 0);
    return hipGetLastError();
}

}  // namespace moed
