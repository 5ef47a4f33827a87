// Internal interface of the prompt-side calls: C ABI (prompt.hip) to kernels, and what prompt.hip needs of moedecode.hip.
#pragma once

#include "launch.h"

namespace moed {

// MOED_OK, or MOED_ERR_HIP with the error kept for moed_last_hip_error() (moedecode.hip).
int abi_status(hipError_t e);
// Under MOED_CHECK the input check of a call (moedecode.hip); MOED_OK otherwise. gate_up, down: those scales are folded
// into a conversion to bfloat16.
int abi_check(const CheckArgs& c, bool gate_up, bool down, hipStream_t s);
// Residual addition and root-mean-square norm (norm.hip). res: 0 no residual, 1 bfloat16, 2 float32.
constexpr int kNormMaxH = 32768;              // a row stays in the registers of one workgroup
constexpr int kMaxTokens = 1 << 22;           // tokens of a prompt-side call: one workgroup each in a launch's 2^32 threads
struct NormArgs {
    const void* x;          // [B][H] bf16 or f32
    const void* residual;   // [B][H] or null
    const void* gain;       // [H]
    void* residual_out;     // null: the sum is not stored
    void* out;              // null: MXFP8 only
    uint8_t* q;             // [B][H] codes or null
    uint8_t* q_s;           // [B][H/32]
    int B, H;
    float eps;
    bool gain_bf16, out_bf16;
};
hipError_t launch_norm(const NormArgs& p, bool x_bf16, int res, hipStream_t s);
// Slots sorted by expert (group.hip). counts: group_workspace(n, E) bytes.
constexpr int kGroupOneBlock = 8192;          // slots one workgroup sorts by itself
constexpr int kGroupMaxE = 2048;
size_t group_workspace(int n, int E);
hipError_t launch_group(const int32_t* ids, int n, int E, int32_t* counts, int32_t* order, int32_t* position,
                        int32_t* offsets, hipStream_t s);
// Weighted sum of each token's expert rows (combine.hip).
struct CombineArgs {
    const void* y;          // [R][H] bf16 or f32
    const int32_t* position;// [B][k]
    const float* w;         // [B][k]
    void* out;              // [B][H]
    int B, k, H, R;
    bool out_bf16;
};
hipError_t launch_combine(const CombineArgs& p, bool y_bf16, hipStream_t s);
// Products grouped by expert over ragged rows (product.hip and the files it calls). The rows of
// expert e are offsets[e] .. offsets[e+1]-1; u_q set: SiLU(w row) * (u row).
constexpr int kOutBF16 = 0, kOutF32 = 1, kOutMX8 = 2;
struct ProductArgs {
    const void* a;          // [n_a][K] bf16, or E4M3 codes with a_s
    const uint8_t* a_s;     // [n_a][K/32] (null: bf16)
    const int32_t* order;   // [R]: row r reads a[order[r] / k]; null: a[r]
    const int32_t* offsets; // [E+1]
    const uint8_t *w_q, *w_s, *u_q, *u_s;   // [E][N][K] codes (K/2 bytes a row for MXFP4), [E][N][K/32]
    void* out;              // [R][N] bf16, f32 or E4M3 codes
    uint8_t* out_s;         // [R][N/32] (MXFP8 out)
    int n_a, k, R, E, K, N;
    uint32_t inv_k;         // 2^32 / k (2^32 - 1 for k = 1)
    int s_row;              // bytes between rows of scales: a multiple of 4, at least 16
    bool fp4;               // weights are MXFP4
    bool fast;              // MXFP8 rows, rounded outputs: on the scaled matrix instructions
    int out_kind;           // kOutBF16, kOutF32 or kOutMX8
};
// The kernels fetch block scales 16 bytes of a row at a time, from dword
// addresses. Where rows of K/32 bytes are shorter or no multiple of 4, they are
// first copied to `scales` with rows of a multiple of 16 (product_scales_bytes;
// 0: not needed).
size_t product_scales_bytes(int E, int K, int N, int n_a, bool mx_rows, bool two);
hipError_t launch_product(ProductArgs p, void* scales, hipStream_t s);
// avg: rows an expert on average.
hipError_t launch_product_bf16(const ProductArgs& p, int avg, hipStream_t s);
hipError_t launch_product_mx(const ProductArgs& p, int avg, hipStream_t s);
hipError_t launch_product_exact(const ProductArgs& p, int avg, hipStream_t s);
hipError_t launch_product_rounded(const ProductArgs& p, int avg, hipStream_t s);

}  // namespace moed
