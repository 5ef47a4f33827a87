// Products grouped by expert where experts have few rows (decode batches, the
// tails of small prompts): every weight is read once for up to 16*MT rows, so
// the kernel is bound by the weight stream.
//
// A workgroup takes one tile of rows of one expert and NF fragments of 16
// weight rows; its four wavefronts split K (steps of 128 values, dealt in
// turn), which keeps four times as many loads in flight as one wavefront per
// fragment would, and their sums are added through LDS in wavefront order.
// Weights go straight from memory to the registers of the one lane that
// multiplies them; rows come from L2.
#include "product_common.h"

namespace moed {

namespace {

constexpr int kFewWaves = 4;

// One lane's operands of a 128-value step. Values at k >= K are zero.
struct Step {
    u32x4 lo, hi;           // E4M3: 16 codes each; E2M1: lo only
    uint32_t s;             // scale byte
};

template <bool FP4, bool SPLIT>
__device__ __forceinline__ Step load_codes(const uint8_t* row, const uint8_t* scales, int k0, int g, int K)
{
    // SPLIT: the E4M3 layout of the scaled matrix instruction (two runs of 16
    // codes 64 apart); otherwise the 32 codes of block g
    Step r;
    r.lo = u32x4{0, 0, 0, 0};
    r.hi = u32x4{0, 0, 0, 0};
    r.s = 0;
    if constexpr (FP4) {
        if (k0 + 32 * g < K)
            r.lo = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(row + k0 / 2 + 16 * g));
    } else {
        const int a = SPLIT ? k0 + 16 * g : k0 + 32 * g, b = SPLIT ? a + 64 : a + 16;
        if (a < K)
            r.lo = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(row + a));
        if (b < K)
            r.hi = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(row + b));
    }
    if (k0 + 32 * g < K)
        r.s = scales[k0 / 32 + g];
    return r;
}

__device__ __forceinline__ i32x8 as_operand(const Step& s)
{
    return i32x8{(int)s.lo.x, (int)s.lo.y, (int)s.lo.z, (int)s.lo.w, (int)s.hi.x, (int)s.hi.y, (int)s.hi.z, (int)s.hi.w};
}

template <bool FP4>
__device__ __forceinline__ bf16x8 decode_quarter(const Step& s, float scale, int q)
{
    if constexpr (FP4) {
        return decode8_scaled_fp4(s.lo[q], scale);
    } else {
        const u32x4 v = q < 2 ? s.lo : s.hi;
        return decode8_scaled((q & 1) ? u32x2{v.z, v.w} : u32x2{v.x, v.y}, scale);
    }
}

}  // namespace

// MX: rows in MXFP8 (else bfloat16). NF fragments of 16 weight rows; with GLU
// the first half are gate rows and the second half the same up rows.
template <bool MX, bool FP4, bool GLU, int OUT, int NF, int MT>
__global__ void __launch_bounds__(kFewWaves * kWave)
moe_product_few_kernel(ProductArgs p)
{
    constexpr int kOutFrags = GLU ? NF / 2 : NF;
    constexpr int kNeurons = 16 * kOutFrags;
    extern __shared__ __align__(16) int lds[];
    f32x4* part = reinterpret_cast<f32x4*>(lds);                  // [wave][MT][NF][64]
    const TileList tl = tile_list(lds + kFewWaves * MT * NF * kWave * 4, p.E);
    __shared__ int wsum[kFewWaves];
    const int tid = threadIdx.x, lane = tid % kWave, w = tid / kWave;
    const int g = lane / 16, col = lane % 16;
    const int tiles = build_tiles<kFewWaves * kWave>(tl, p.offsets, p.E, p.R, 16 * MT, wsum);
    const int nblk = (p.N + kNeurons - 1) / kNeurons;
    const long long items = (long long)tiles * nblk;
    const int steps = (p.K + 127) / 128;
    const size_t code_row = FP4 ? (size_t)p.K / 2 : (size_t)p.K, scale_row = (size_t)p.K / 32;
    const int wg = xcd_contiguous(blockIdx.x, gridDim.x);

    for (long long item = wg; item < items; item += gridDim.x) {
        const int tile = (int)(item / nblk), n0 = (int)(item % nblk) * kNeurons;
        const int e = tile_expert(tl, p.E, tile);
        if (e >= p.E)
            continue;                                             // uniform
        const int m0 = (tile - tl.first[e]) * (16 * MT), rows = tl.n[e];
        if (m0 < 0 || m0 >= rows)
            continue;
        // this lane's weight rows and row pointers (rows behind the tile's last repeat it)
        const uint8_t* wq[NF];
        const uint8_t* ws[NF];
#pragma unroll
        for (int f = 0; f < NF; ++f) {
            const bool up = GLU && f >= NF / 2;
            int n = n0 + 16 * (up ? f - NF / 2 : f) + col;
            n = n < p.N ? n : p.N - 1;
            const size_t row = (size_t)e * (size_t)p.N + (size_t)n;
            wq[f] = (up ? p.u_q : p.w_q) + row * code_row;
            ws[f] = (up ? p.u_s : p.w_s) + row * scale_row;
        }
        const uint8_t* aq[MT];
        const uint8_t* as[MT];
        int src[MT];
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            int r = m0 + 16 * t + col;
            r = tl.lo[e] + (r < rows ? r : rows - 1);
            src[t] = source_row(p, r);
            const size_t from = (size_t)(src[t] < 0 ? 0 : src[t]);
            aq[t] = static_cast<const uint8_t*>(p.a) + from * (size_t)p.K * (MX ? 1 : 2);
            as[t] = MX ? p.a_s + from * scale_row : nullptr;
        }
        f32x4 acc[MT][NF];
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int f = 0; f < NF; ++f)
                acc[t][f] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        for (int st = w; st < steps; st += kFewWaves) {
            const int k0 = st * 128;
            Step wc[NF];
#pragma unroll
            for (int f = 0; f < NF; ++f)
                wc[f] = load_codes<FP4, MX>(wq[f], ws[f], k0, g, p.K);
            if constexpr (MX) {
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    const Step ac = load_codes<false, true>(aq[t], as[t], k0, g, p.K);
#pragma unroll
                    for (int f = 0; f < NF; ++f)
                        acc[t][f] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                            as_operand(wc[f]), as_operand(ac), acc[t][f], FP4 ? 4 : 0, 0, 0, (int)wc[f].s, 0, (int)ac.s);
                }
            } else {
                float sc[NF];
#pragma unroll
                for (int f = 0; f < NF; ++f)
                    sc[f] = ue8m0_to_f32(wc[f].s);
                u32x4 x[MT][4];
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        x[t][q] = k0 + 32 * g < p.K
                                      ? *reinterpret_cast<const u32x4*>(aq[t] + 2 * (size_t)(k0 + 32 * g + 8 * q))
                                      : u32x4{0, 0, 0, 0};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
#pragma unroll
                    for (int f = 0; f < NF; ++f) {
                        const bf16x8 wv = decode_quarter<FP4>(wc[f], sc[f], q);
#pragma unroll
                        for (int t = 0; t < MT; ++t)
                            acc[t][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                wv, __builtin_bit_cast(bf16x8, x[t][q]), acc[t][f], 0, 0, 0);
                    }
                }
            }
        }
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int f = 0; f < NF; ++f)
                part[((w * MT + t) * NF + f) * kWave + lane] = acc[t][f];
        __syncthreads();
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            if (t % kFewWaves != w)
                continue;                                         // whole wavefronts
            f32x4 y[NF];
#pragma unroll
            for (int f = 0; f < NF; ++f) {
                y[f] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int q = 0; q < kFewWaves; ++q)
                    y[f] += part[((q * MT + t) * NF + f) * kWave + lane];
            }
            f32x4 o[kOutFrags];
#pragma unroll
            for (int f = 0; f < kOutFrags; ++f)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float v = y[f][i];
                    if constexpr (GLU)
                        v = swiglu(v, y[f + NF / 2][i]);
                    o[f][i] = src[t] < 0 ? __builtin_nanf("") : v;
                }
            const int r = m0 + 16 * t + col;
            store_row<OUT>(p, tl.lo[e] + r, n0, g, r < rows, o);
        }
        __syncthreads();                                          // part is written again by the next item
    }
}

namespace {

template <bool MX, bool FP4, bool GLU, int OUT, int MT>
hipError_t launch_few(const ProductArgs& p, hipStream_t s)
{
    constexpr int NF = GLU && OUT == kOutMX8 ? 4 : 2;
    constexpr int kNeurons = 16 * (GLU ? NF / 2 : NF);
    const size_t lds = (size_t)kFewWaves * MT * NF * kWave * 16 + tile_list_bytes(p.E);
    const void* f = reinterpret_cast<const void*>(&moe_product_few_kernel<MX, FP4, GLU, OUT, NF, MT>);
    if (lds > 65536)
        if (hipError_t e = set_max_dynamic_lds(f, (int)lds))
            return e;
    const long long tiles = (long long)p.R / (16 * MT) + (p.R < p.E ? p.R : p.E);
    long long grid = tiles * ((p.N + kNeurons - 1) / kNeurons);
    grid = grid < 1 ? 1 : grid > 2048 ? 2048 : grid;
    hipLaunchKernelGGL((moe_product_few_kernel<MX, FP4, GLU, OUT, NF, MT>), dim3((unsigned)grid), dim3(kFewWaves * kWave),
                       lds, s, p);
    return hipGetLastError();
}

template <bool MX, bool FP4, bool GLU, int OUT>
hipError_t few_rows(const ProductArgs& p, int mt, hipStream_t s)
{
    if (mt <= 1)
        return launch_few<MX, FP4, GLU, OUT, 1>(p, s);
    if (mt == 2)
        return launch_few<MX, FP4, GLU, OUT, 2>(p, s);
    return launch_few<MX, FP4, GLU, OUT, 4>(p, s);
}

template <bool MX, bool FP4>
hipError_t few_out(const ProductArgs& p, int mt, hipStream_t s)
{
    if (p.u_q) {
        if (p.out_kind == kOutBF16)
            return few_rows<MX, FP4, true, kOutBF16>(p, mt, s);
        if (p.out_kind == kOutF32)
            return few_rows<MX, FP4, true, kOutF32>(p, mt, s);
        return few_rows<MX, FP4, true, kOutMX8>(p, mt, s);
    }
    if (p.out_kind == kOutBF16)
        return few_rows<MX, FP4, false, kOutBF16>(p, mt, s);
    return few_rows<MX, FP4, false, kOutF32>(p, mt, s);
}

}  // namespace

hipError_t launch_product_few(const ProductArgs& p, int row_tiles, hipStream_t s)
{
    if (p.a_s)
        return p.fp4 ? few_out<true, true>(p, row_tiles, s) : few_out<true, false>(p, row_tiles, s);
    return p.fp4 ? few_out<false, true>(p, row_tiles, s) : few_out<false, false>(p, row_tiles, s);
}

// The rows per expert that the host can know are an average: R over the
// experts that can have any.
hipError_t launch_product(const ProductArgs& p, hipStream_t s)
{
    const int experts = p.R < p.E ? p.R : p.E;
    const long long avg = ((long long)p.R + experts - 1) / experts;
    if (avg > 32)
        return launch_product_tiled(p, (int)avg, s);
    return launch_product_few(p, avg <= 16 ? 1 : avg <= 32 ? 2 : 4, s);
}

}  // namespace moed
