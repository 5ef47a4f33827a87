// Shared parts of the products grouped by expert over ragged rows: the list of
// row tiles, the sources of rows, and the store of a tile.
//
// The matrix instructions take the weights as the A operand and the rows as the
// B operand, so a lane receives four consecutive outputs of one row.
//
// MXFP8 rows on the scaled instructions: v_mfma_scale_f32_16x16x128_f8f6f4, codes
// and block scales as they are stored, products and block scales exact, float32
// accumulators; of eight neighbouring products what lies 2^-14 below the largest
// is dropped. Lane l supplies row l%16; with g = l/16 its E4M3 codes are
// k = 16g..16g+15 and 64+16g..64+16g+15, its E2M1 codes k = 32g..32g+31, and its
// scale byte is the one of block k = 32g..32g+31. It receives rows 4g..4g+3 of
// column l%16.
// Otherwise: v_mfma_f32_16x16x32_bf16 on BF16 rows, or MXFP8 rows decoded to it,
// and weights decoded to BF16, with their block scales folded into the
// conversion (exact for scale codes 10..245 of MXFP8 and 2..252 of MXFP4).
#pragma once

#include "grouped_common.h"
#include "mx_encode.h"
#include "prompt.h"

namespace moed {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// first[e] = row tiles of the experts before e and begin[e] = first row of e
// (E + 1 ints of LDS each), built by every workgroup. Offsets are clamped into
// [0, R] and made to rise, so garbage in them leads to wrong rows but to no
// access outside. Returns all tiles. All threads must call it; ends with a
// barrier.
template <int THREADS>
__device__ __forceinline__ int build_tiles(int* first, int* begin, const int32_t* offsets, int E, int R, int tile_rows,
                                           int* wsum)
{
    constexpr int W = THREADS / kWave;
    const int tid = threadIdx.x, lane = tid % kWave, w = tid / kWave;
    int done = 0, top = 0;                                    // tiles and largest offset so far
    for (int e0 = 0; e0 <= E; e0 += THREADS) {                // begin[e] = the largest of offsets[0..e], clamped
        const int e = e0 + tid;
        int lo = e <= E ? offsets[e] : 0;
        lo = lo < 0 ? 0 : lo > R ? R : lo;
#pragma unroll
        for (int d = 1; d < kWave; d <<= 1) {
            const int o = __shfl_up(lo, d);
            lo = lane >= d && o > lo ? o : lo;
        }
        if (lane == kWave - 1)
            wsum[w] = lo;
        __syncthreads();
        int all = top;
        lo = top > lo ? top : lo;
#pragma unroll
        for (int q = 0; q < W; ++q) {
            lo = q < w && wsum[q] > lo ? wsum[q] : lo;
            all = wsum[q] > all ? wsum[q] : all;
        }
        if (e <= E)
            begin[e] = lo;
        top = all;
        __syncthreads();
    }
    for (int e0 = 0; e0 < E; e0 += THREADS) {
        const int e = e0 + tid;
        const int tiles = e < E ? (begin[e + 1] - begin[e] + tile_rows - 1) / tile_rows : 0;
        int inc = tiles;
#pragma unroll
        for (int d = 1; d < kWave; d <<= 1) {
            const int o = __shfl_up(inc, d);
            if (lane >= d)
                inc += o;
        }
        if (lane == kWave - 1)
            wsum[w] = inc;
        __syncthreads();
        int before = done, all = 0;
#pragma unroll
        for (int q = 0; q < W; ++q) {
            before += q < w ? wsum[q] : 0;
            all += wsum[q];
        }
        if (e < E)
            first[e] = before + inc - tiles;
        done += all;
        __syncthreads();
    }
    if (tid == 0)
        first[E] = done;
    __syncthreads();
    return done;
}

// Expert of a global tile: the number of experts whose tiles all come before it.
__device__ __forceinline__ int tile_expert(const int* first, int E, int tile)
{
    const int lane = threadIdx.x % kWave;
    int e = 0;
    for (int base = 0; base < E; base += kWave) {
        const unsigned long long m = __ballot(base + lane < E && first[base + lane + 1] <= tile);
        e += __popcll(m);
        if (m != ~0ull)
            break;
    }
    return __builtin_amdgcn_readfirstlane(e);
}

// Row of `a` that a slot of an order reads: slot / k, -1 where that lies outside.
__device__ __forceinline__ int source_row(const ProductArgs& p, int slot)
{
    // slot / k by the reciprocal 2^32 / k, off by at most one
    int q = (int)__umulhi((unsigned)slot, p.inv_k);
    const int rest = slot - q * p.k;
    q += rest >= p.k ? 1 : rest < 0 ? -1 : 0;
    return slot < 0 || q >= p.n_a ? -1 : q;
}

// Largest of v over the four lane groups (lanes with equal lane % 16).
__device__ __forceinline__ uint32_t max_over_groups(uint32_t v)
{
    const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = a[0] > a[1] ? a[0] : a[1];
    const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return b[0] > b[1] ? b[0] : b[1];
}

// Stores 16 rows (m .. m+15 of the expert whose rows begin at row0) of NF
// fragments: lane (col, g) holds outputs n + 16f + 4g .. +3 of row m + col in
// o[f]. They go through `mine` (LDS of this wavefront alone, rows of `stride`
// bytes), so that neighbouring lanes store neighbouring 16-byte pieces of a row
// and lines are written whole. For MXFP8 the fragments 2f and 2f+1 are a block.
template <int OUT, int NF>
__device__ __forceinline__ void store_tile_rows(const ProductArgs& p, uint8_t* mine, int stride, int row0, int m, int rows,
                                                int n, f32x4 (&o)[NF])
{
    constexpr int kBytes = OUT == kOutBF16 ? 2 : 1;
    constexpr int kPieces = NF * kBytes;                      // 16-byte pieces of a row
    const int lane = threadIdx.x % kWave, g = lane / 16, col = lane % 16;
    uint8_t* at = mine + col * stride;
    if constexpr (OUT == kOutF32) {                           // 16 bytes a lane as they are
        if (m + col < rows) {
            float* out = static_cast<float*>(p.out) + (size_t)(row0 + m + col) * (size_t)p.N + (size_t)(n + 4 * g);
#pragma unroll
            for (int f = 0; f < NF; ++f)
                if (n + 16 * f < p.N)
                    *reinterpret_cast<f32x4*>(out + 16 * f) = o[f];
        }
        return;
    }
    if constexpr (OUT == kOutMX8) {
        static_assert(NF % 2 == 0, "whole blocks");
#pragma unroll
        for (int f = 0; f < NF; f += 2) {
            uint32_t a = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t u = __float_as_uint(o[f][i]) & 0x7FFFFFFFu, v = __float_as_uint(o[f + 1][i]) & 0x7FFFFFFFu;
                a = u > a ? u : a;
                a = v > a ? v : a;
            }
            a = max_over_groups(a);
            const uint32_t c = mx8_scale_code(a);
            *reinterpret_cast<uint32_t*>(at + 16 * f + 4 * g) = mx8_codes4(o[f][0], o[f][1], o[f][2], o[f][3], c);
            *reinterpret_cast<uint32_t*>(at + 16 * f + 16 + 4 * g) =
                mx8_codes4(o[f + 1][0], o[f + 1][1], o[f + 1][2], o[f + 1][3], c);
            if (g == 0 && m + col < rows && n + 16 * f < p.N)
                p.out_s[((size_t)(row0 + m + col) * (size_t)p.N + (size_t)n) / 32 + f / 2] = (uint8_t)c;
        }
    } else {
#pragma unroll
        for (int f = 0; f < NF; ++f) {
            uint32_t* q = reinterpret_cast<uint32_t*>(at + (16 * f + 4 * g) * 2);
            q[0] = f32x2_to_bf16x2_rne(o[f][0], o[f][1]);
            q[1] = f32x2_to_bf16x2_rne(o[f][2], o[f][3]);
        }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int i = 0; i < (16 * kPieces + kWave - 1) / kWave; ++i) {
        const int piece = i * kWave + lane, r = piece / kPieces, c = piece % kPieces;
        if (r < 16 && m + r < rows && n + c * (16 / kBytes) < p.N) {
            const u32x4 v = *reinterpret_cast<const u32x4*>(mine + r * stride + 16 * c);
            uint8_t* out = static_cast<uint8_t*>(p.out) + ((size_t)(row0 + m + r) * (size_t)p.N + (size_t)n) * kBytes + 16 * c;
            *reinterpret_cast<u32x4*>(out) = v;
        }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

}  // namespace moed
