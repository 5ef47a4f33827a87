// Shared parts of the products grouped by expert over ragged rows
// (product_few.hip, product_tiled.hip): the list of row tiles, the operands of
// one step of the matrix instructions, and the store of a tile.
//
// The matrix instructions take the weights as the A operand and the rows as the
// B operand, so a lane receives four consecutive outputs of one row.
//
// MXFP8 rows: v_mfma_scale_f32_16x16x128_f8f6f4, codes and block scales as they
// are stored, products and block scales exact, float32 accumulators. Lane l
// supplies row l%16; with g = l/16 its E4M3 codes are k = 16g..16g+15 and
// 64+16g..64+16g+15, its E2M1 codes k = 32g..32g+31, and its scale byte is the
// one of block k = 32g..32g+31. It receives rows 4g..4g+3 of column l%16.
// BF16 rows: v_mfma_f32_16x16x32_bf16 on weights decoded to BF16 with their
// block scale folded into the conversion (exact for scale codes 10..245 of
// MXFP8 and 2..252 of MXFP4).
#pragma once

#include "grouped_common.h"

namespace moed {

typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kProductMaxE = 2048;

// Row tiles of all experts, built by every workgroup in its LDS: first[e] =
// tiles of the experts before e, lo[e] = first row, n[e] = rows. Offsets are
// clamped into [0, R], so garbage in them leads to wrong rows but to no access
// outside, and the total is capped at what any valid offsets can give. All
// threads must call it; ends with a barrier.
struct TileList {
    int* first;             // E + 1
    int* lo;                // E
    int* n;                 // E
};

inline size_t tile_list_bytes(int E) { return ((size_t)3 * E + 1) * 4; }

__device__ __forceinline__ TileList tile_list(int* lds, int E)
{
    return TileList{lds, lds + E + 1, lds + 2 * E + 1};
}

template <int THREADS>
__device__ __forceinline__ int build_tiles(const TileList& t, const int32_t* offsets, int E, int R, int tile_rows,
                                           int* wsum)
{
    constexpr int W = THREADS / kWave;
    const int tid = threadIdx.x, lane = tid % kWave, w = tid / kWave;
    int done = 0;
    for (int e0 = 0; e0 < E; e0 += THREADS) {
        const int e = e0 + tid;
        int lo = 0, hi = 0;
        if (e < E) {
            lo = offsets[e];
            hi = offsets[e + 1];
            lo = lo < 0 ? 0 : lo > R ? R : lo;
            hi = hi < lo ? lo : hi > R ? R : hi;
        }
        const int tiles = (hi - lo + tile_rows - 1) / tile_rows;
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
        if (e < E) {
            t.first[e] = before + inc - tiles;
            t.lo[e] = lo;
            t.n[e] = hi - lo;
        }
        done += all;
        __syncthreads();
    }
    if (tid == 0)
        t.first[E] = done;
    __syncthreads();
    const int most = R / tile_rows + (R < E ? R : E);
    return done < 0 ? 0 : done < most ? done : most;
}

// Expert of a global tile: the number of experts whose tiles all come before it.
__device__ __forceinline__ int tile_expert(const TileList& t, int E, int tile)
{
    const int lane = threadIdx.x % kWave;
    int e = 0;
    for (int base = 0; base < E; base += kWave) {
        const unsigned long long m = __ballot(base + lane < E && t.first[base + lane + 1] <= tile);
        e += __popcll(m);
        if (m != ~0ull)
            break;
    }
    return __builtin_amdgcn_readfirstlane(e);
}

// Source row in `a` of sorted row r; -1 where order[r] lies outside.
__device__ __forceinline__ int source_row(const ProductArgs& p, int r)
{
    if (!p.order)
        return r;
    const int t = p.order[r];
    const int s = t < 0 ? -1 : t / p.k;
    return s < p.n_a ? s : -1;
}

// Stores NF fragments of 4 consecutive outputs of row r: fragment f holds
// outputs n0 + 16f + 4g .. +3 (g = lane / 16). For MXFP8 the fragments 2f and
// 2f+1 of the four lane groups are one block. All 64 lanes must call it.
template <int OUT, int NF>
__device__ __forceinline__ void store_row(const ProductArgs& p, int r, int n0, int g, bool valid, f32x4 (&y)[NF])
{
    const size_t at = (size_t)r * (size_t)p.N + (size_t)(n0 + 4 * g);
    if constexpr (OUT == kOutMX8) {
#pragma unroll
        for (int f = 0; f < NF; f += 2) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t a = __float_as_uint(y[f][i]) & 0x7FFFFFFFu;
                const uint32_t b = __float_as_uint(y[f + 1][i]) & 0x7FFFFFFFu;
                m = a > m ? a : m;
                m = b > m ? b : m;
            }
            const uint32_t o = (uint32_t)__shfl_xor((int)m, 16);
            m = o > m ? o : m;
            const uint32_t q = (uint32_t)__shfl_xor((int)m, 32);
            m = q > m ? q : m;
            const uint32_t c = mx8_scale_code(m);
            if (valid && n0 + 16 * f < p.N) {
                uint8_t* out = static_cast<uint8_t*>(p.out) + at + 16 * f;
                *reinterpret_cast<uint32_t*>(out) = mx8_codes4(y[f][0], y[f][1], y[f][2], y[f][3], c);
                *reinterpret_cast<uint32_t*>(out + 16) = mx8_codes4(y[f + 1][0], y[f + 1][1], y[f + 1][2], y[f + 1][3], c);
                if (g == 0)
                    p.out_s[((size_t)r * (size_t)p.N + (size_t)n0) / 32 + f / 2] = (uint8_t)c;
            }
        }
    } else {
#pragma unroll
        for (int f = 0; f < NF; ++f) {
            if (valid && n0 + 16 * f < p.N) {
                if constexpr (OUT == kOutBF16)
                    *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(p.out) + at + 16 * f) =
                        u32x2{f32x2_to_bf16x2_rne(y[f][0], y[f][1]), f32x2_to_bf16x2_rne(y[f][2], y[f][3])};
                else
                    *reinterpret_cast<f32x4*>(static_cast<float*>(p.out) + at + 16 * f) = y[f];
            }
        }
    }
}

}  // namespace moed
