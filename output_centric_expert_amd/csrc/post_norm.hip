// The end of a block and the norm in front of the next one:
//   t = y * rsqrt(mean(y^2) + post_eps) * post_gain        (y without post_gain)
//   s = residual_scale * residual + scale * act(gate) * t;  residual_out = s, rounded
//   out = s * rsqrt(mean(s^2) + eps) * gain, rounded once, and in MXFP8 by the rule of norm.hip
// y is given, or is the weighted sum of a token's expert rows (combine.hip), which then is never stored: each of its
// k rows is read, the sum goes on in registers. Everything between loads and stores is float32.
//
// A row stays in the registers of its threads (8 values a piece, NV pieces a thread, TPR threads a row) from the loads to
// the last store; two sums over the row stand between them. All loads are asked for in front of the first use of any
// (raw: a conversion behind a load waits for it), so that a row waits for memory once, twice where its rows' places
// come first. Memory bound: 8192 tokens of 4096 values, bfloat16, with MXFP8 55-59 us (5.1-5.5 TB/s), 8 expert rows a token of
// 2048 and a float32 residual 76-78 us (5.6 TB/s; 105 with conversions between the loads), rows of 1111 values 24 us (3 TB/s:
// their pieces begin at any element, and their stores do not fill lines); one token 3-4 us, two round trips and the launch.
// Rows may begin at any element and have any length: a piece that would pass the row's end is the row's last 8 values
// instead, of which the first `skip` are another piece's: loaded, but neither counted nor stored.
#include "activation.h"
#include "mx_encode.h"
#include "row_values.h"

namespace moed {

namespace {

// Where a thread's piece lies in the row.
struct Piece {
    int at, skip;
    bool mine;
};

__device__ __forceinline__ Piece piece_of(int h, int H)
{
    if (H < 8)
        return {0, 0, h == 0};
    const int last = H - 8;
    return {h < last ? h : last, h < last ? 0 : h - last, h < H};
}

template <bool NT>
__device__ __forceinline__ Raw load_piece(bool bf16, const void* p, size_t row, const Piece& piece, int H)
{
    return H < 8 ? load_short(bf16, p, row, H) : load_raw<NT>(bf16, p, row + piece.at);     // rows shorter than a piece
}

__device__ __forceinline__ void store_piece(bool bf16, void* p, size_t row, const Piece& piece, int H, const float (&v)[8])
{
    if (H % 8 == 0) {                                         // whole pieces at 16-byte borders: streaming
        if (bf16)
            store_vals<true>(p, row + piece.at, v);
        else
            store_vals<false>(p, row + piece.at, v);
        return;
    }
    if (piece.skip == 0 && H >= 8) {
        if (bf16)
            store_any<true>(p, row + piece.at, 8, v);
        else
            store_any<false>(p, row + piece.at, 8, v);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (H < 8 ? i < H : i >= piece.skip) {
            const size_t at = row + (H < 8 ? 0 : piece.at) + i;
            if (bf16)
                static_cast<uint16_t*>(p)[at] = f32_to_bf16_rne(v[i]);
            else
                static_cast<float*>(p)[at] = v[i];
        }
}

__device__ __forceinline__ float gate_value(float g, int act)
{
    return act == kActSigmoid ? sigmoid(g) : act == kActTanh ? tanh_of(g) : g;
}

// 1 / sqrt(mean of squares + eps) of a row as mul * scale: mul is 1 but for rows whose squares would underflow
// (kSmall), which are taken times kLift.
struct Root {
    float mul, scale;
};

template <int NV, int WAVES>
__device__ __forceinline__ Root row_root(const float (&s)[NV][8], int H, float eps, float* part)
{
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int v = 0; v < 8; ++v)
            ss = __builtin_fmaf(s[i][v], s[i][v], ss);
    ss = row_sum<WAVES>(ss, part);
    float mul = 1.0f;
    if (eps < kSmall && ss < kSmall) {            // the same for all threads of a row
        mul = kLift;
        eps = eps * kLift * kLift;
        ss = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int v = 0; v < 8; ++v)
                ss = __builtin_fmaf(s[i][v] * kLift, s[i][v] * kLift, ss);
        if constexpr (WAVES > 1)
            __syncthreads();                      // everybody has the first sum
        ss = row_sum<WAVES>(ss, part);
    }
    return {mul, rsqrtf(ss / (float)H + eps)};
}

}  // namespace

template <int NV, int TPR, bool YBF16, bool RBF16, bool ROWS>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR)
moe_post_norm_kernel(PostNormArgs p)
{
    constexpr int kRows = TPR < 256 ? 256 / TPR : 1;          // rows per workgroup
    constexpr int kWaves = TPR / kWave;
    constexpr int kAhead = NV > 2 ? 2 : YBF16 ? 8 : 4;        // expert rows asked for before the first is added
    __shared__ float part[2][kWaves];
    const int t = threadIdx.x % TPR;
    const long long b = (long long)blockIdx.x * kRows + (kRows > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x / TPR) : 0);
    if (b >= p.B)
        return;                                               // whole wavefronts; no barrier follows for kRows > 1
    const int H = p.H;
    const size_t row = (size_t)b * (size_t)H;
    const float token_gate = p.gate_shape == kGateToken
        ? (p.gate_bf16 ? bf16_val(static_cast<const uint16_t*>(p.gate)[b]) : static_cast<const float*>(p.gate)[b]) : 0.0f;
    Piece piece[NV];
    Raw r[NV], y[NV], gate[NV], post_gain[NV], gain[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        piece[i] = piece_of((t + i * TPR) * 8, H);
        if (piece[i].mine) {
            if constexpr (!ROWS)
                y[i] = load_piece<true>(YBF16, p.y, row, piece[i], H);
            r[i] = load_piece<true>(RBF16, p.residual, row, piece[i], H);
        }
    }
    auto load_gains = [&](int i) {
        if (p.gate_shape == kGateFull)
            gate[i] = load_piece<true>(p.gate_bf16, p.gate, row, piece[i], H);
        else if (p.gate_shape == kGateChannel)
            gate[i] = load_piece<false>(p.gate_bf16, p.gate, 0, piece[i], H);
        if (p.post_gain)
            post_gain[i] = load_piece<false>(p.post_gain_bf16, p.post_gain, 0, piece[i], H);
        if (p.gain)
            gain[i] = load_piece<false>(p.gain_bf16, p.gain, 0, piece[i], H);
    };
    // Where a thread has two pieces, gates and gains come late: their registers would cost workgroups on a CU (8192 tokens
    // of 4096 values, gate of each value: 74 us with everything early, 66 with the gate alone).
    constexpr bool kEarly = NV == 1;
    float s[NV][8];
    if constexpr (ROWS) {
        const int32_t* pos = p.position + (size_t)b * p.k;
        const float* w = p.topk_w + (size_t)b * p.k;
        bool bad = false;
        for (int j = 0; j < p.k; ++j)
            bad |= (unsigned)pos[j] >= (unsigned)p.R;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
            for (int v = 0; v < 8; ++v)
                s[i][v] = 0.0f;
            if (!piece[i].mine)
                continue;
            if (bad) {                                        // the token's outputs are NaN, and no row is read
#pragma unroll
                for (int v = 0; v < 8; ++v)
                    s[i][v] = __builtin_nanf("");
                continue;
            }
            for (int j0 = 0; j0 < p.k; j0 += kAhead) {
                Raw rows[kAhead];
#pragma unroll
                for (int j = 0; j < kAhead; ++j)
                    if (j0 + j < p.k)                         // uniform over the row
                        rows[j] = load_piece<true>(YBF16, p.y, (size_t)pos[j0 + j] * (size_t)H, piece[i], H);
#pragma unroll
                for (int j = 0; j < kAhead; ++j)
                    if (j0 + j < p.k) {
                        float one[8];
                        raw_values(YBF16, rows[j], one);
#pragma unroll
                        for (int v = 0; v < 8; ++v)
                            s[i][v] = __builtin_fmaf(w[j0 + j], one[v], s[i][v]);
                    }
            }
        }
        if constexpr (kEarly)
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (piece[i].mine)
                    load_gains(i);
    } else {
        if constexpr (kEarly)
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (piece[i].mine)
                    load_gains(i);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            raw_values(YBF16, y[i], s[i]);
            if (!piece[i].mine)
#pragma unroll
                for (int v = 0; v < 8; ++v)
                    s[i][v] = 0.0f;
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)                              // values of other pieces
#pragma unroll
        for (int v = 0; v < 7; ++v)
            s[i][v] = v < piece[i].skip ? 0.0f : s[i][v];
    Root post = {1.0f, 1.0f};
    if (p.post_gain)
        post = row_root<NV, kWaves>(s, H, p.post_eps, part[0]);
    const float one_gate = p.gate_shape == kGateToken ? p.scale * gate_value(token_gate, p.gate_act) : p.scale;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (!piece[i].mine)
            continue;
        if constexpr (!kEarly)
            load_gains(i);
        if (p.post_gain) {
            float g[8];
            raw_values(p.post_gain_bf16, post_gain[i], g);
#pragma unroll
            for (int v = 0; v < 8; ++v)
                s[i][v] = s[i][v] * post.mul * post.scale * g[v];
        }
        float g[8], held[8];
        raw_values(RBF16, r[i], held);
#pragma unroll
        for (int v = 0; v < 8; ++v)
            g[v] = one_gate;
        if (p.gate_shape >= kGateChannel) {
            raw_values(p.gate_bf16, gate[i], g);
            if (p.gate_act != kActNone)
#pragma unroll
                for (int v = 0; v < 8; ++v)
                    g[v] = gate_value(g[v], p.gate_act);
#pragma unroll
            for (int v = 0; v < 8; ++v)
                g[v] *= p.scale;
        }
#pragma unroll
        for (int v = 0; v < 8; ++v)
            s[i][v] = v < piece[i].skip || (H < 8 && v >= H)
                ? 0.0f : __builtin_fmaf(p.residual_scale, held[v], g[v] * s[i][v]);
        if (p.residual_out)
            store_piece(RBF16, p.residual_out, row, piece[i], H, s[i]);
    }
    if (!p.gain)
        return;
    const Root pre = row_root<NV, kWaves>(s, H, p.eps, part[1]);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (!piece[i].mine)
            continue;
        float o[8];
        raw_values(p.gain_bf16, gain[i], o);
#pragma unroll
        for (int v = 0; v < 8; ++v)
            o[v] = s[i][v] * pre.mul * pre.scale * o[v];
        if (p.out)
            store_piece(p.out_bf16, p.out, row, piece[i], H, o);
        if (p.q) {                                            // H is a multiple of 32: four whole lanes per block
            uint32_t m = 0;
#pragma unroll
            for (int v = 0; v < 8; ++v) {
                const uint32_t a = __float_as_uint(o[v]) & 0x7FFFFFFFu;
                m = a > m ? a : m;
            }
            m = quad_max(m);
            u32x2 codes;
            const uint32_t c = mx8_scale_code(m);
            codes.x = mx8_codes4(o[0], o[1], o[2], o[3], c);
            codes.y = mx8_codes4(o[4], o[5], o[6], o[7], c);
            __builtin_nontemporal_store(codes, reinterpret_cast<u32x2*>(p.q + row + piece[i].at));
            if ((t & 3) == 0)
                p.q_s[(row + piece[i].at) / 32] = (uint8_t)c;
        }
    }
}

namespace {

template <int NV, int TPR>
hipError_t launch_shape(const PostNormArgs& p, bool y_bf16, bool r_bf16, hipStream_t s)
{
    constexpr int kRows = TPR < 256 ? 256 / TPR : 1;
    const dim3 grid((unsigned)((p.B + kRows - 1) / kRows)), block(TPR < 256 ? 256 : TPR);
#define MOED_POST(Y, R) \
    do { \
        if (p.position) hipLaunchKernelGGL((moe_post_norm_kernel<NV, TPR, Y, R, true>), grid, block, 0, s, p); \
        else hipLaunchKernelGGL((moe_post_norm_kernel<NV, TPR, Y, R, false>), grid, block, 0, s, p); \
    } while (0)
    if (y_bf16) {
        if (r_bf16) MOED_POST(true, true);
        else MOED_POST(true, false);
    } else {
        if (r_bf16) MOED_POST(false, true);
        else MOED_POST(false, false);
    }
#undef MOED_POST
    return hipGetLastError();
}

}  // namespace

hipError_t launch_post_norm(const PostNormArgs& p, bool y_bf16, bool residual_bf16, hipStream_t s)
{
    if (p.H <= 512)
        return launch_shape<1, 64>(p, y_bf16, residual_bf16, s);
    if (p.H <= 1024)
        return launch_shape<2, 64>(p, y_bf16, residual_bf16, s);
    if (p.H <= 2048)
        return launch_shape<1, 256>(p, y_bf16, residual_bf16, s);
    // few rows: more threads a row (one token of 4096 values 3.6 us, with 256 threads 4.3; 512 tokens 6.2 and 6.7, 8192 of
    // 4095 values 65.6 and 59.4)
    if (p.H <= 4096 && p.B < 512)
        return launch_shape<1, 512>(p, y_bf16, residual_bf16, s);
    if (p.H <= 4096)
        return launch_shape<2, 256>(p, y_bf16, residual_bf16, s);
    if (p.H <= 8192)
        return launch_shape<2, 512>(p, y_bf16, residual_bf16, s);
    if (p.H <= 16384)
        return launch_shape<2, 1024>(p, y_bf16, residual_bf16, s);
    return launch_shape<4, 1024>(p, y_bf16, residual_bf16, s);
}

}  // namespace moed
