// Products grouped by expert where experts have many rows (prompts): tiles of
// rows x weight rows through LDS, matrix instructions on what it holds.
#include "product_common.h"

namespace moed {

namespace {

// How rows enter the matrix instructions.
constexpr int kRowsBF16 = 0;      // bfloat16 rows, weights decoded to bfloat16
constexpr int kRowsMX = 1;        // MXFP8 rows and MX weights as stored, scaled matrix instructions
constexpr int kRowsMXExact = 2;   // MXFP8 rows and weights both decoded to bfloat16

__device__ const u32x4 kZeros = {0, 0, 0, 0};     // source of the values behind the end of a row

// 16 bytes per lane from global memory straight to LDS: lane i of the wavefront
// writes base + 16 i (base uniform). No register receives the data; the caller
// waits on vmcnt before a barrier. Written as asm because the compiler makes
// every later LDS read wait for the builtin's load, whatever buffer it fills.
// (m0 is set by each; nothing else in these kernels uses it.)
__device__ __forceinline__ void load_to_lds16(const void* src, uint32_t base)
{
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(src), "s"(base) : "memory");
}

__device__ __forceinline__ void load_to_lds4(const void* src, uint32_t base)
{
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off" ::"v"(src), "s"(base) : "memory");
}

template <int ROWS, bool FP4, int RT, int NT, int WR, int WN>
struct Shape {
    static constexpr bool kMX = ROWS == kRowsMX;
    static constexpr int kThreads = WR * WN * kWave;
    static constexpr int kBM = 16 * RT * WR;                  // rows of a tile
    static constexpr int kBN = 16 * NT * WN;                  // weight rows of a tile
    static constexpr int kBK = kMX ? 128 : 64;                // values of a step
    static constexpr int kRU = ROWS == kRowsMXExact ? 4 : 8;  // 16-byte units of a row and step
    static constexpr int kWU = kBK / (FP4 ? 32 : 16);         // ... of a weight row and step
    static constexpr int kRowLoads = kBM * kRU / kThreads;
    static constexpr int kWLoads = kBN * kWU / kThreads;
    static constexpr int kRowBytes = kBM * kRU * 16, kWBytes = kBN * kWU * 16;
    static constexpr int kBufBytes = kRowBytes + kWBytes;
    // block scales of 128 values: one dword per row and weight row
    static constexpr int kScaleRows = kBN + (ROWS != kRowsBF16 ? kBM : 0);
    static constexpr int kScaleLoads = (kScaleRows + kThreads - 1) / kThreads;
    static constexpr int kScaleBytes = kScaleLoads * kThreads * 4;
    static constexpr int kLds = 2 * kBufBytes + 2 * kScaleBytes;
    static_assert(kBM * kRU % kThreads == 0 && kBN * kWU % kThreads == 0, "whole loads per thread");
    static_assert((kThreads / kRU) % 8 == 0 && (kThreads / kWU) % 8 == 0, "a thread's loads share their place in the row");
};

// Units of a row are stored at c ^ swizzle(row), so that the lanes that read one
// unit of 8 (or 16) neighbouring rows together meet different banks.
template <int UNITS>
__device__ __forceinline__ int swizzle(int row)
{
    return UNITS == 8 ? row & 7 : UNITS == 4 ? (row >> 1) & 3 : (row >> 2) & 1;
}

}  // namespace

template <int ROWS, bool FP4, bool GLU, int OUT, int RT, int NT, int WR, int WN>
__global__ void __launch_bounds__(WR * WN * kWave)
moe_product_tiled_kernel(ProductArgs p, int nblk, int group_blocks, int aligned_scales)
{
    using S = Shape<ROWS, FP4, RT, NT, WR, WN>;
    constexpr bool kMX = S::kMX;
    constexpr int kOutFrags = GLU ? NT / 2 : NT;
    constexpr int kNeurons = 16 * kOutFrags * WN;             // outputs of a tile
    extern __shared__ __align__(16) uint8_t lds[];
    uint32_t* const scales = reinterpret_cast<uint32_t*>(lds + 2 * S::kBufBytes);   // [2][kScaleBytes / 4]
    const TileList tl = tile_list(reinterpret_cast<int*>(lds + S::kLds), p.E);
    __shared__ int wsum[WR * WN];
    const int tid = threadIdx.x, lane = tid % kWave;
    const int w = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int g = lane / 16, col = lane % 16;
    const int wr = w / WN, wn = w % WN;
    const int tiles = build_tiles<S::kThreads>(tl, p.offsets, p.E, p.R, S::kBM, wsum);
    const long long items = (long long)tiles * nblk;
    const int steps = (p.K + S::kBK - 1) / S::kBK;
    const size_t w_row = FP4 ? (size_t)p.K / 2 : (size_t)p.K, s_row = (size_t)p.K / 32;
    const size_t a_row = ROWS == kRowsBF16 ? 2 * (size_t)p.K : (size_t)p.K;
    const uint32_t lds0 = (uint32_t)(size_t)(__attribute__((address_space(3))) uint8_t*)lds;

    for (long long item = xcd_contiguous(blockIdx.x, gridDim.x); item < items; item += gridDim.x) {
        // items of one expert are neighbours; within it blocks of weight rows in
        // groups, so that a group's weights and the expert's rows meet in one L2
        const int e = tile_expert(tl, p.E, (int)(item / nblk));
        if (e >= p.E)
            continue;                                         // uniform
        const int mt = tl.first[e + 1] - tl.first[e];
        const long long local = item - (long long)tl.first[e] * nblk;
        const int grp = (int)(local / ((long long)group_blocks * mt));
        const int rest = (int)(local - (long long)grp * group_blocks * mt);
        const int in_grp = nblk - grp * group_blocks < group_blocks ? nblk - grp * group_blocks : group_blocks;
        const int n0 = (grp * group_blocks + rest % in_grp) * kNeurons;
        const int m0 = (rest / in_grp) * S::kBM;
        const int rows = tl.n[e], row0 = tl.lo[e];
        if (m0 < 0 || m0 >= rows || n0 >= p.N)
            continue;                                         // only for offsets that decrease

        // sources of this thread's loads (rows behind the last repeat it)
        const uint8_t* rsrc[S::kRowLoads];
        const uint8_t* wsrc[S::kWLoads];
        const int rc = (tid % S::kRU) ^ swizzle<S::kRU>(tid / S::kRU);      // unit within the row and step
        const int wc = (tid % S::kWU) ^ swizzle<S::kWU>(tid / S::kWU);
#pragma unroll
        for (int i = 0; i < S::kRowLoads; ++i) {
            int r = m0 + i * (S::kThreads / S::kRU) + tid / S::kRU;
            r = r < rows ? r : rows - 1;
            const int src = source_row(p, row0 + r);
            rsrc[i] = static_cast<const uint8_t*>(p.a) + (size_t)(src < 0 ? 0 : src) * a_row + 16 * rc;
        }
        auto weight_row = [&](int rr, bool& up) {             // weight row of place rr of the tile
            const int wv = rr / (16 * NT), f = rr / 16 % NT;
            up = GLU && f >= NT / 2;
            const int n = n0 + (wv * kOutFrags + (up ? f - NT / 2 : f)) * 16 + rr % 16;
            return (size_t)e * (size_t)p.N + (size_t)(n < p.N ? n : p.N - 1);
        };
#pragma unroll
        for (int i = 0; i < S::kWLoads; ++i) {
            bool up;
            const size_t n = weight_row(i * (S::kThreads / S::kWU) + tid / S::kWU, up);
            wsrc[i] = (up ? p.u_q : p.w_q) + n * w_row + 16 * wc;
        }
        const uint8_t* ssrc[S::kScaleLoads];
#pragma unroll
        for (int i = 0; i < S::kScaleLoads; ++i) {
            const int rr = i * S::kThreads + tid;
            if (rr < S::kBN) {
                bool up;
                const size_t n = weight_row(rr, up);
                ssrc[i] = (up ? p.u_s : p.w_s) + n * s_row;
            } else {
                int r = m0 + (rr - S::kBN);
                r = r < rows ? r : rows - 1;
                const int src = ROWS != kRowsBF16 ? source_row(p, row0 + r) : 0;
                ssrc[i] = (ROWS != kRowsBF16 ? p.a_s : p.w_s) + (size_t)(src < 0 ? 0 : src) * s_row;
            }
        }

        auto stage = [&](int st) {
            const uint32_t buf = lds0 + (uint32_t)(st & 1) * S::kBufBytes + (uint32_t)w * 1024u;
            const int k0 = st * S::kBK;
            if (k0 + S::kBK <= p.K) {
#pragma unroll
                for (int i = 0; i < S::kRowLoads; ++i)
                    load_to_lds16(rsrc[i] + (size_t)st * (S::kRU * 16), buf + i * S::kThreads * 16);
#pragma unroll
                for (int i = 0; i < S::kWLoads; ++i)
                    load_to_lds16(wsrc[i] + (size_t)st * (S::kWU * 16), buf + S::kRowBytes + i * S::kThreads * 16);
            } else {                                          // the last step of a K that is no multiple of kBK
                const bool rin = k0 + rc * (S::kBK / S::kRU) < p.K, win = k0 + wc * (S::kBK / S::kWU) < p.K;
#pragma unroll
                for (int i = 0; i < S::kRowLoads; ++i)
                    load_to_lds16(rin ? rsrc[i] + (size_t)st * (S::kRU * 16) : reinterpret_cast<const uint8_t*>(&kZeros),
                                  buf + i * S::kThreads * 16);
#pragma unroll
                for (int i = 0; i < S::kWLoads; ++i)
                    load_to_lds16(win ? wsrc[i] + (size_t)st * (S::kWU * 16) : reinterpret_cast<const uint8_t*>(&kZeros),
                                  buf + S::kRowBytes + i * S::kThreads * 16);
            }
            if (kMX || (st & 1) == 0) {                       // scales of 128 values
                const int q = kMX ? st : st / 2;
                if (aligned_scales) {
#pragma unroll
                    for (int i = 0; i < S::kScaleLoads; ++i)
                        load_to_lds4(ssrc[i] + 4 * (size_t)q, lds0 + 2 * S::kBufBytes + (q & 1) * S::kScaleBytes +
                                                                  (uint32_t)(i * S::kThreads + w * kWave) * 4u);
                } else {
#pragma unroll
                    for (int i = 0; i < S::kScaleLoads; ++i) {
                        uint32_t v = 0;
#pragma unroll
                        for (int b = 0; b < 4; ++b)
                            if (128 * q + 32 * b < p.K)
                                v |= (uint32_t)ssrc[i][4 * (size_t)q + b] << (8 * b);
                        scales[(q & 1) * (S::kScaleBytes / 4) + i * S::kThreads + tid] = v;
                    }
                }
            }
        };

        f32x4 acc[RT][NT];
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int f = 0; f < NT; ++f)
                acc[r][f] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

        __syncthreads();                                      // the last item's readers of both buffers are done
        stage(0);
        for (int st = 0; st < steps; ++st) {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            __syncthreads();                                  // step st is in LDS; the other buffer is free
            if (st + 1 < steps)
                stage(st + 1);
            const uint8_t* rb = lds + (st & 1) * S::kBufBytes;
            const uint8_t* wb = rb + S::kRowBytes;
            const int q = kMX ? st : st / 2;
            const uint8_t* sb = reinterpret_cast<const uint8_t*>(scales) + (q & 1) * S::kScaleBytes;
            const int sbyte = kMX ? g : 2 * (st & 1) + g / 2;
            auto unit = [&](const uint8_t* base, int units, int row, int c) {
                const int sw = units == 8 ? swizzle<8>(row) : units == 4 ? swizzle<4>(row) : swizzle<2>(row);
                return *reinterpret_cast<const u32x4*>(base + (row * units + (c ^ sw)) * 16);
            };
            if constexpr (kMX) {
                i32x8 wv[NT];
                int wsc[NT];
#pragma unroll
                for (int f = 0; f < NT; ++f) {
                    const int row = (wn * NT + f) * 16 + col;
                    const u32x4 lo = unit(wb, S::kWU, row, g);
                    const u32x4 hi = FP4 ? u32x4{0, 0, 0, 0} : unit(wb, S::kWU, row, 4 + g);
                    wv[f] = i32x8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
                    wsc[f] = sb[row * 4 + sbyte];
                }
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    const int row = (wr * RT + r) * 16 + col;
                    const u32x4 lo = unit(rb, 8, row, g), hi = unit(rb, 8, row, 4 + g);
                    const i32x8 av{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
                    const int asc = sb[(S::kBN + row) * 4 + sbyte];
#pragma unroll
                    for (int f = 0; f < NT; ++f)
                        acc[r][f] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wv[f], av, acc[r][f], FP4 ? 4 : 0, 0,
                                                                                     0, wsc[f], 0, asc);
                }
            } else {
                // lane group g multiplies values 16g .. 16g+15 of the step, 8 per matrix instruction
                bf16x8 wv[NT][2];
#pragma unroll
                for (int f = 0; f < NT; ++f) {
                    const int row = (wn * NT + f) * 16 + col;
                    const float sc = ue8m0_to_f32(sb[row * 4 + sbyte]);
                    if constexpr (FP4) {
                        const u32x2 c = *reinterpret_cast<const u32x2*>(
                            wb + (row * 2 + ((g / 2) ^ swizzle<2>(row))) * 16 + 8 * (g % 2));
                        wv[f][0] = decode8_scaled_fp4(c.x, sc);
                        wv[f][1] = decode8_scaled_fp4(c.y, sc);
                    } else {
                        const u32x4 c = unit(wb, 4, row, g);
                        wv[f][0] = decode8_scaled(u32x2{c.x, c.y}, sc);
                        wv[f][1] = decode8_scaled(u32x2{c.z, c.w}, sc);
                    }
                }
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    const int row = (wr * RT + r) * 16 + col;
                    bf16x8 av[2];
                    if constexpr (ROWS == kRowsMXExact) {
                        const float sc = ue8m0_to_f32(sb[(S::kBN + row) * 4 + sbyte]);
                        const u32x4 c = unit(rb, 4, row, g);
                        av[0] = decode8_scaled(u32x2{c.x, c.y}, sc);
                        av[1] = decode8_scaled(u32x2{c.z, c.w}, sc);
                    } else {
                        av[0] = __builtin_bit_cast(bf16x8, unit(rb, 8, row, 2 * g));
                        av[1] = __builtin_bit_cast(bf16x8, unit(rb, 8, row, 2 * g + 1));
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int f = 0; f < NT; ++f)
                            acc[r][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv[f][h], av[h], acc[r][f], 0, 0, 0);
                }
            }
        }

#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const int m = m0 + (wr * RT + r) * 16 + col;
            const bool valid = m < rows;
            const int at = row0 + (valid ? m : rows - 1);
            const bool bad = source_row(p, at) < 0;
            f32x4 o[kOutFrags];
#pragma unroll
            for (int f = 0; f < kOutFrags; ++f)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float v = acc[r][f][i];
                    if constexpr (GLU)
                        v = swiglu(v, acc[r][f + NT / 2][i]);
                    o[f][i] = bad ? __builtin_nanf("") : v;
                }
            store_row<OUT>(p, at, n0 + wn * kOutFrags * 16, g, valid, o);
        }
    }
}

namespace {

template <int ROWS, bool FP4, bool GLU, int OUT, int RT, int NT, int WR, int WN>
hipError_t launch_shape(const ProductArgs& p, hipStream_t s)
{
    using S = Shape<ROWS, FP4, RT, NT, WR, WN>;
    constexpr int kNeurons = 16 * (GLU ? NT / 2 : NT) * WN;
    const size_t lds = S::kLds + tile_list_bytes(p.E);
    const void* f = reinterpret_cast<const void*>(&moe_product_tiled_kernel<ROWS, FP4, GLU, OUT, RT, NT, WR, WN>);
    if (lds > 65536)
        if (hipError_t e = set_max_dynamic_lds(f, (int)lds))
            return e;
    const int nblk = (p.N + kNeurons - 1) / kNeurons;
    const long long tiles = (long long)p.R / S::kBM + (p.R < p.E ? p.R : p.E);
    const int per_cu = (int)((size_t)163840 / lds);
    long long grid = tiles * nblk;
    const long long most = 256LL * (per_cu < 1 ? 1 : per_cu > 4 ? 4 : per_cu);
    grid = grid < most ? grid : most;
    const bool aligned = (p.K / 32) % 4 == 0 && ((uintptr_t)p.w_s & 3) == 0 && (!p.u_s || ((uintptr_t)p.u_s & 3) == 0) &&
                         (!p.a_s || ((uintptr_t)p.a_s & 3) == 0);
    // weight rows of about 2 MiB per group of blocks
    const long long bytes = (long long)S::kBN * p.K / (FP4 ? 2 : 1);
    long long group = (2LL << 20) / bytes;
    group = group < 1 ? 1 : group > nblk ? nblk : group;
    hipLaunchKernelGGL((moe_product_tiled_kernel<ROWS, FP4, GLU, OUT, RT, NT, WR, WN>), dim3((unsigned)grid),
                       dim3(S::kThreads), lds, s, p, nblk, (int)group, aligned ? 1 : 0);
    return hipGetLastError();
}

template <int ROWS, bool FP4, bool GLU, int OUT>
hipError_t tiled_shape(const ProductArgs& p, int avg, hipStream_t s)
{
    if constexpr (ROWS == kRowsMX) {
        if (avg >= 256)
            return launch_shape<ROWS, FP4, GLU, OUT, 8, 4, 2, 4>(p, s);   // 256 x 256
        return launch_shape<ROWS, FP4, GLU, OUT, 4, 4, 2, 2>(p, s);       // 128 x 128
    } else {
        if (avg >= 96)
            return launch_shape<ROWS, FP4, GLU, OUT, 4, 4, 2, 2>(p, s);   // 128 x 128
        return launch_shape<ROWS, FP4, GLU, OUT, 4, 4, 1, 4>(p, s);       // 64 x 256
    }
}

template <bool FP4>
hipError_t tiled_rows(const ProductArgs& p, int avg, hipStream_t s)
{
    if (p.u_q) {
        if (!p.a_s) {
            if (p.out_kind == kOutBF16)
                return tiled_shape<kRowsBF16, FP4, true, kOutBF16>(p, avg, s);
            if (p.out_kind == kOutF32)
                return tiled_shape<kRowsBF16, FP4, true, kOutF32>(p, avg, s);
            return tiled_shape<kRowsBF16, FP4, true, kOutMX8>(p, avg, s);
        }
        if (p.out_kind == kOutBF16)
            return tiled_shape<kRowsMX, FP4, true, kOutBF16>(p, avg, s);
        if (p.out_kind == kOutF32)
            return tiled_shape<kRowsMXExact, FP4, true, kOutF32>(p, avg, s);
        return tiled_shape<kRowsMX, FP4, true, kOutMX8>(p, avg, s);
    }
    if (!p.a_s)
        return p.out_kind == kOutBF16 ? tiled_shape<kRowsBF16, FP4, false, kOutBF16>(p, avg, s)
                                      : tiled_shape<kRowsBF16, FP4, false, kOutF32>(p, avg, s);
    return p.out_kind == kOutBF16 ? tiled_shape<kRowsMX, FP4, false, kOutBF16>(p, avg, s)
                                  : tiled_shape<kRowsMXExact, FP4, false, kOutF32>(p, avg, s);
}

}  // namespace

hipError_t launch_product_tiled(const ProductArgs& p, int avg, hipStream_t s)
{
    return p.fp4 ? tiled_rows<true>(p, avg, s) : tiled_rows<false>(p, avg, s);
}

}  // namespace moed
