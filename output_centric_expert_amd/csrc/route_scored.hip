// Router by scores, a bias for balance and groups of experts:
//   s_e = softmax(l)_e or sigmoid(l_e), rounded to float32;  c_e = s_e + bias[e] in float32
//   the topk_group groups of the largest value (largest c, or the float32 sum of the two largest)
//   the k experts of the largest c in them; weights s (over their sum + 1e-20) * routed_scale
//
// Scores are computed in float64 and rounded once, so that what is compared does not depend on how exp is computed: a
// float32 exp differs by an ulp from one program to the next, and of some thousand tokens of 256 experts a few have
// two choices that close. Float64 runs at the rate of float32 on this card's vector unit.
//
// L lanes own a token, NPL neighbouring experts each (expert = lane * NPL + t), so that among equal keys the lowest
// lane, and in it the lowest t, is the lowest expert. A key is the order-preserving map of the choice to 32 bits; 0: not
// to be chosen. What bounds it is the vector unit with many tokens (16384 of 256 experts, 8 of 4 of 8 groups: 14.3-15.2 us a
// call in a graph, 13.4 of calls that overlap, for 1411 instructions a wavefront, which are 9.4 us of issue; its bytes are
// 3), one round trip to memory and the rounds' chain with few (1 token of 128 experts 4.1 us, 64 of 256 5.4). So there are
// two kernels:
//  - few tokens, many experts or k: a token a wavefront. Round j takes the largest key of the lanes (DPP), the lowest
//    lane that holds it writes the expert to the token's list in LDS and clears its key.
//  - many tokens: 16 lanes a token, four tokens a wavefront. Key and expert are packed into one float64 (43 bits, the lower
//    expert the larger), which one instruction compares; a lane sorts its own, keeps eight, and four exchanges with other
//    lanes leave the token's best eight in order in every one.
#include "block.h"
#include "lds_loads.h"
#include "mx_encode.h"
#include "row_values.h"

namespace moed {

namespace {

constexpr int kRouteWaves = 4;

// Order-preserving map of a float32 to 32 bits; -0 as +0. No finite number or infinity maps to 0.
__device__ __forceinline__ uint32_t order_key(float v)
{
    const uint32_t u = __float_as_uint(v + 0.0f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

__device__ __forceinline__ float key_value(uint32_t key)
{
    return __uint_as_float((key & 0x80000000u) ? (key & 0x7FFFFFFFu) : ~key);
}

// Key of a choice: 0 for NaN and -infinity.
__device__ __forceinline__ uint32_t choice_key(float c) { return c > -__builtin_inff() ? order_key(c) : 0u; }

// exp(x) for |x| up to 150 (callers clamp it there: a float32 score is 0 or 1 beyond): 2^n times Taylor's series of the
// rest below ln(2)/2, whose first term left out is 2^-52 of it. n is rounded by adding 1.5 * 2^52, which leaves it in
// the low word, and goes into the exponent by an addition: conversions have a quarter of the rate.
__device__ __forceinline__ double exp64(double x)
{
    const double shifted = __builtin_fma(x, 0x1.71547652b82fep+0, 0x1.8p52), n = shifted - 0x1.8p52;
    double r = __builtin_fma(-n, 0x1.62e42fefa39efp-1, x);
    r = __builtin_fma(-n, 0x1.abc9e3b39803fp-56, r);
    double p = 1.0 / 479001600.0;
    p = __builtin_fma(p, r, 1.0 / 39916800.0);
    p = __builtin_fma(p, r, 1.0 / 3628800.0);
    p = __builtin_fma(p, r, 1.0 / 362880.0);
    p = __builtin_fma(p, r, 1.0 / 40320.0);
    p = __builtin_fma(p, r, 1.0 / 5040.0);
    p = __builtin_fma(p, r, 1.0 / 720.0);
    p = __builtin_fma(p, r, 1.0 / 120.0);
    p = __builtin_fma(p, r, 1.0 / 24.0);
    p = __builtin_fma(p, r, 1.0 / 6.0);
    p = __builtin_fma(p, r, 0.5);
    p = __builtin_fma(p, r, 1.0);
    p = __builtin_fma(p, r, 1.0);
    const uint64_t u = __builtin_bit_cast(uint64_t, p);
    const uint32_t high = (uint32_t)(u >> 32) + ((uint32_t)__builtin_bit_cast(uint64_t, shifted) << 20);
    return __builtin_bit_cast(double, (uint64_t)high << 32 | (uint32_t)u);
}

// 1 / d for normal d: the hardware's estimate (2^-23 at least) and one step of third order.
__device__ __forceinline__ double reciprocal64(double d)
{
    const double y = __builtin_amdgcn_rcp(d), e = __builtin_fma(-d, y, 1.0);
    return __builtin_fma(y, __builtin_fma(e, e, e), y);
}

// v of another lane of the row of 16.
template <int CTRL>
__device__ __forceinline__ uint32_t from_lane(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}

template <int CTRL>
__device__ __forceinline__ double from_lane(double v)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(double, (uint64_t)from_lane<CTRL>((uint32_t)(u >> 32)) << 32 | from_lane<CTRL>((uint32_t)u));
}

constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kMirror8 = 0x141, kMirror16 = 0x140;      // DPP: quad_perm, row_half_mirror, row_mirror

template <int CTRL>
__device__ __forceinline__ uint32_t max_dpp32(uint32_t v)
{
    const uint32_t o = from_lane<CTRL>(v);
    return o > v ? o : v;
}

// Largest v of the L lanes of a token, in each of them.
template <int L>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v)
{
    v = max_dpp32<kXor1>(v);
    v = max_dpp32<kXor2>(v);
    v = max_dpp32<kMirror8>(v);
    v = max_dpp32<kMirror16>(v);
    if constexpr (L == 64) {
        const uint32_t a = (uint32_t)__builtin_amdgcn_readlane((int)v, 0), b = (uint32_t)__builtin_amdgcn_readlane((int)v, 16);
        const uint32_t c = (uint32_t)__builtin_amdgcn_readlane((int)v, 32), d = (uint32_t)__builtin_amdgcn_readlane((int)v, 48);
        const uint32_t e = a > b ? a : b, f = c > d ? c : d;
        v = e > f ? e : f;
    }
    return v;
}

// Sum over the L lanes of a token, the same bits in each of them (partners add the same two numbers).
template <int L>
__device__ __forceinline__ double lanes_sum(double v)
{
    v += from_lane<kXor1>(v);
    v += from_lane<kXor2>(v);
    v += from_lane<kMirror8>(v);
    v += from_lane<kMirror16>(v);
    if constexpr (L == 64) {
        v += __shfl_xor(v, 16);
        v += __shfl_xor(v, 32);
    }
    return v;
}

// Lowest lane of the token (0 .. L-1) among those of the ballot, -1 for none.
template <int L>
__device__ __forceinline__ int first_lane(unsigned long long ballot, int lane)
{
    if constexpr (L == 64)
        return __ffsll(ballot) - 1;
    return __ffs((int)((uint32_t)(ballot >> (lane & ~(L - 1))) & ((1u << L) - 1u))) - 1;
}

// This lane's experts and what they are worth.
template <int NPL>
struct Experts {
    float score[NPL];
    uint32_t key[NPL];
};

template <int L, int NPL, bool BF16>
__device__ __forceinline__ void score_experts(const RouteArgs& p, size_t b, int tl, Experts<NPL>& x)
{
    float l[NPL], bias[NPL];
    const float nan = __builtin_nanf("");
    const int e0 = tl * NPL;
    const bool whole = NPL % 4 == 0 && e0 + NPL <= p.E;
    const size_t at = b * (size_t)p.E + e0;
#pragma unroll
    for (int t = 0; t < NPL; ++t)
        bias[t] = 0.0f;
    if (whole) {
        if constexpr (NPL % 4 == 0) {
#pragma unroll
            for (int t = 0; t < NPL; t += 4) {
                if constexpr (BF16) {
                    typedef u32x2 u32x2_at2 __attribute__((aligned(2)));
                    const u32x2 u = *reinterpret_cast<const u32x2_at2*>(static_cast<const uint16_t*>(p.logits) + at + t);
                    l[t] = bf16_lo(u.x);
                    l[t + 1] = bf16_hi(u.x);
                    l[t + 2] = bf16_lo(u.y);
                    l[t + 3] = bf16_hi(u.y);
                } else {
                    const f32x4 u = ld_at4<false>(static_cast<const float*>(p.logits) + at + t);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        l[t + i] = u[i];
                }
            }
            if (p.bias) {
#pragma unroll
                for (int t = 0; t < NPL; t += 4) {
                    const f32x4 u = ld_at4<false>(p.bias + e0 + t);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        bias[t + i] = u[i];
                }
            }
        }
    } else {
#pragma unroll
        for (int t = 0; t < NPL; ++t) {
            l[t] = nan;
            if (p.bias && e0 + t < p.E)
                bias[t] = p.bias[e0 + t];
            if (e0 + t < p.E)
                l[t] = BF16 ? bf16_val(static_cast<const uint16_t*>(p.logits)[at + t]) : static_cast<const float*>(p.logits)[at + t];
        }
    }
    if (p.sigmoid) {
#pragma unroll
        for (int t = 0; t < NPL; ++t)
            x.score[t] = (float)reciprocal64(1.0 + exp64((double)__builtin_amdgcn_fmed3f(-l[t], -150.0f, 150.0f)));
    } else {
        float m = -__builtin_inff();
#pragma unroll
        for (int t = 0; t < NPL; ++t)
            m = l[t] > m ? l[t] : m;
        m = key_value(lanes_max<L>(order_key(m)));
        double ex[NPL], sum = 0.0;
#pragma unroll
        for (int t = 0; t < NPL; ++t) {
            ex[t] = l[t] != l[t] ? 0.0 : l[t] == m ? 1.0 : exp64(__builtin_fmax((double)l[t] - (double)m, -150.0));
            sum += ex[t];
        }
        sum = reciprocal64(lanes_sum<L>(sum));
#pragma unroll
        for (int t = 0; t < NPL; ++t)
            x.score[t] = (float)(ex[t] * sum);
    }
#pragma unroll
    for (int t = 0; t < NPL; ++t) {
        const float c = x.score[t] + bias[t];                 // without a bias: exactly the score
        x.key[t] = l[t] == l[t] ? choice_key(c) : 0u;
    }
}

// The sum (or the larger) of a group's two largest choices, as a key.
__device__ __forceinline__ uint32_t group_key(bool top2, uint32_t k1, uint32_t k2)
{
    if (!top2 || k2 == 0u)
        return k1;
    const uint32_t sum = choice_key(key_value(k1) + key_value(k2));
    return sum ? sum : 1u;                                    // an overflow to -infinity stays above "none"
}

__device__ __forceinline__ void keep_two(uint32_t v, uint32_t& k1, uint32_t& k2)
{
    const uint32_t low = v < k1 ? v : k1;
    k1 = v > k1 ? v : k1;
    k2 = low > k2 ? low : k2;
}

template <int CTRL>
__device__ __forceinline__ void merge_two(uint32_t& k1, uint32_t& k2)
{
    const uint32_t o1 = from_lane<CTRL>(k1), o2 = from_lane<CTRL>(k2);
    keep_two(o1, k1, k2);
    k2 = o2 > k2 ? o2 : k2;
}

// Clears the keys of experts whose group is not among the best. words: this token's L * NPL words of LDS.
template <int L, int NPL>
__device__ __forceinline__ void choose_groups(const RouteArgs& p, int lane, int tl, uint32_t* words, uint32_t (&key)[NPL])
{
    const int size = p.E / p.n_group, lanes = size / NPL;
    // a group is whole lanes, 1, 2, 4, 8 or 16 of them: its value without LDS, in its first lane
    const bool aligned = size % NPL == 0 && lanes <= 16 && (lanes & (lanes - 1)) == 0;
    uint32_t worth = 0;
    int per = 1;                                              // lanes from one group's value to the next
    if (aligned) {
        uint32_t k1 = 0, k2 = 0;
#pragma unroll
        for (int t = 0; t < NPL; ++t)
            keep_two(key[t], k1, k2);
        if (lanes > 1)
            merge_two<kXor1>(k1, k2);
        if (lanes > 2)
            merge_two<kXor2>(k1, k2);
        if (lanes > 4)
            merge_two<kMirror8>(k1, k2);
        if (lanes > 8)
            merge_two<kMirror16>(k1, k2);
        per = lanes;
        worth = tl % lanes == 0 ? group_key(p.top2, k1, k2) : 0u;
    } else {
#pragma unroll
        for (int t = 0; t < NPL; ++t)
            words[tl * NPL + t] = key[t];
        wave_lds_fence();
        if (tl < p.n_group) {
            uint32_t k1 = 0, k2 = 0;
            int at = tl % size;                               // lanes begin at different banks
            for (int i = 0; i < size; ++i) {
                keep_two(words[tl * size + at], k1, k2);
                at = at + 1 == size ? 0 : at + 1;
            }
            worth = group_key(p.top2, k1, k2);
        }
    }
    unsigned long long taken = 0;                             // by the lane that has the group's value
    for (int j = 0; j < p.topk_group; ++j) {
        const uint32_t m = lanes_max<L>(worth);
        const int win = first_lane<L>(__ballot(worth == m && m != 0u), lane);
        if (win >= 0)
            taken |= 1ull << win;
        if (tl == win)
            worth = 0;
    }
    if (aligned) {
        const bool keep = (taken >> (tl - tl % per)) & 1ull;
#pragma unroll
        for (int t = 0; t < NPL; ++t)
            key[t] = keep ? key[t] : 0u;
    } else {
        int g = tl * NPL / size, left = size - (tl * NPL - g * size);
#pragma unroll
        for (int t = 0; t < NPL; ++t) {
            key[t] = (taken >> (g & 63)) & 1ull ? key[t] : 0u;
            if (--left == 0) {
                left = size;
                ++g;
            }
        }
    }
}

// What a token's lanes write: slot j of each lane's, the score it was chosen with.
template <int L>
__device__ __forceinline__ void store_slots(const RouteArgs& p, size_t b, int tl, int chosen, const int* picks, const float* scores,
                                            bool live = true)
{
    double sum = 0.0;
    for (int j = tl; j < chosen; j += L)
        sum += (double)scores[picks[j]];
    const double mul = (double)p.routed_scale * (p.renormalize ? reciprocal64(lanes_sum<L>(sum) + 1e-20) : 1.0);
    if (!live)
        return;
    const size_t kt = (size_t)p.k + (size_t)p.n_shared;
    for (int j = tl; j < p.k; j += L) {
        const int e = j < chosen ? picks[j] : -1;
        p.ids[b * kt + j] = e;
        p.w[b * kt + j] = e >= 0 ? (float)((double)scores[e] * mul) : __builtin_nanf("");
    }
    for (int i = tl; i < p.n_shared; i += L) {
        p.ids[b * kt + p.k + i] = p.E + i;
        p.w[b * kt + p.k + i] = 1.0f;
    }
}

}  // namespace

// A token a wavefront.
template <int NPL, bool BF16>
__global__ void __launch_bounds__(kRouteWaves * kWave)
moe_route_scored_kernel(RouteArgs p)
{
    __shared__ uint32_t words[kRouteWaves][kWave * NPL];      // keys for the groups, then scores
    __shared__ int picks[kRouteWaves][kRouteMaxK];
    const int lane = threadIdx.x % kWave, w = threadIdx.x / kWave;
    const long long b = (long long)blockIdx.x * kRouteWaves + w;
    if (b >= p.B)
        return;                                               // whole wavefronts; no barrier follows
    Experts<NPL> x;
    score_experts<kWave, NPL, BF16>(p, (size_t)b, lane, x);
    if (p.topk_group < p.n_group)
        choose_groups<kWave, NPL>(p, lane, lane, words[w], x.key);
    float* const scores = reinterpret_cast<float*>(words[w]);
    wave_lds_fence();
#pragma unroll
    for (int t = 0; t < NPL; ++t)
        scores[lane * NPL + t] = x.score[t];
    uint32_t best = 0;
#pragma unroll
    for (int t = 0; t < NPL; ++t)
        best = x.key[t] > best ? x.key[t] : best;
    int chosen = 0;
    for (int j = 0; j < p.k; ++j) {
        const uint32_t m = lanes_max<kWave>(best);            // uniform
        if (m == 0u)
            break;
        const int win = __ffsll(__ballot(best == m)) - 1;
        chosen = j + 1;
        if (lane == win) {
            int at = 0;
#pragma unroll
            for (int t = NPL - 1; t >= 0; --t)
                at = x.key[t] == m ? t : at;
            best = 0;
#pragma unroll
            for (int t = 0; t < NPL; ++t) {
                x.key[t] = t == at ? 0u : x.key[t];
                best = x.key[t] > best ? x.key[t] : best;
            }
            picks[w][j] = lane * NPL + at;
        }
    }
    wave_lds_fence();
    store_slots<kWave>(p, (size_t)b, lane, chosen, picks[w], scores);
}

namespace {

// Descending order of a and b.
__device__ __forceinline__ void order2(double& a, double& b)
{
    const double high = __builtin_fmax(a, b), low = __builtin_fmin(a, b);
    a = high;
    b = low;
}

// Descending order of v[AT .. AT + N - 1] that rises and falls at most once (a bitonic one).
template <int N, int M>
__device__ __forceinline__ void merge_order(double (&v)[M], int at)
{
    if constexpr (N > 1) {
#pragma unroll
        for (int i = 0; i < N / 2; ++i)
            order2(v[at + i], v[at + i + N / 2]);
        merge_order<N / 2>(v, at);
        merge_order<N / 2>(v, at + N / 2);
    }
}

// Descending order of v[at .. at + N - 1].
template <int N, int M>
__device__ __forceinline__ void sort_order(double (&v)[M], int at)
{
    if constexpr (N > 1) {
        sort_order<N / 2>(v, at);
        sort_order<N / 2>(v, at + N / 2);
#pragma unroll
        for (int i = 0; i < N / 2; ++i)                       // the second half from behind
            order2(v[at + i], v[at + N - 1 - i]);
        merge_order<N / 2>(v, at);
        merge_order<N / 2>(v, at + N / 2);
    }
}

// The largest M of this lane's and another's M, both descending.
template <int CTRL, int M>
__device__ __forceinline__ void merge_lane(double (&v)[M])
{
    double o[M];
#pragma unroll
    for (int i = 0; i < M; ++i)
        o[i] = from_lane<CTRL>(v[i]);
#pragma unroll
    for (int i = 0; i < M; ++i)
        v[i] = __builtin_fmax(v[i], o[M - 1 - i]);
    merge_order<M>(v, 0);
}

constexpr int kManyK = 8;                                     // slots of the kernel for many tokens

}  // namespace

// 16 lanes a token; k at most kManyK, at most 16 groups.
template <int NPL, bool BF16>
__global__ void __launch_bounds__(kRouteWaves * kWave)
moe_route_scored_many_kernel(RouteArgs p)
{
    constexpr int L = 16, TW = kWave / L, kKeep = NPL < kManyK ? NPL : kManyK;
    __shared__ uint32_t words[kRouteWaves * TW][L * NPL];     // keys for the groups, then scores
    __shared__ int picks[kRouteWaves * TW][kManyK];
    const int lane = threadIdx.x % kWave, tl = lane % L, slot = threadIdx.x / L;
    const long long first = ((long long)blockIdx.x * kRouteWaves + threadIdx.x / kWave) * TW;
    if (first >= p.B)
        return;                                               // whole wavefronts; no barrier follows
    const bool live = first + lane / L < p.B;                 // the last wavefront's other lanes repeat the last token
    const size_t b = (size_t)(live ? first + lane / L : p.B - 1);
    Experts<NPL> x;
    score_experts<L, NPL, BF16>(p, b, tl, x);
    if (p.topk_group < p.n_group)
        choose_groups<L, NPL>(p, lane, tl, words[slot], x.key);
    float* const scores = reinterpret_cast<float*>(words[slot]);
    wave_lds_fence();
#pragma unroll
    for (int t = 0; t < NPL; ++t)
        scores[tl * NPL + t] = x.score[t];
    // 2^52 + key * 2^11 + (2^11 - 1 - expert), by its bits: the lower expert is the larger
    double v[NPL];
#pragma unroll
    for (int t = 0; t < NPL; ++t)
        v[t] = __builtin_bit_cast(double, (uint64_t)(0x43300000u | (x.key[t] >> 21)) << 32 |
                                              (x.key[t] << 11 | (uint32_t)(2047 - (tl * NPL + t))));
    double best[kManyK];
    if constexpr (NPL > kManyK) {                             // the best eight of two eights
        sort_order<kManyK>(v, 0);
        sort_order<kManyK>(v, kManyK);
#pragma unroll
        for (int i = 0; i < kManyK; ++i)
            best[i] = __builtin_fmax(v[i], v[2 * kManyK - 1 - i]);
        merge_order<kManyK>(best, 0);
    } else {
        sort_order<NPL>(v, 0);
#pragma unroll
        for (int i = 0; i < kManyK; ++i)
            best[i] = i < kKeep ? v[i < kKeep ? i : 0] : 0x1p52;
    }
    merge_lane<kXor1>(best);
    merge_lane<kXor2>(best);
    merge_lane<kMirror8>(best);
    merge_lane<kMirror16>(best);
    int chosen = 0;
#pragma unroll
    for (int j = 0; j < kManyK; ++j) {
        const uint64_t u = __builtin_bit_cast(uint64_t, best[j]);
        if (j < p.k && (u & 0xFFFFFFFFFF800ull) != 0) {       // a key
            chosen = j + 1;
            if (tl == j)
                picks[slot][j] = 2047 - (int)(u & 2047);
        }
    }
    wave_lds_fence();
    // lanes of no token take part in the sum, and write nothing
    store_slots<L>(p, b, tl, chosen, picks[slot], scores, live);
}

namespace {

template <int NPL>
hipError_t launch_wave(const RouteArgs& p, hipStream_t s)
{
    const dim3 grid((unsigned)((p.B + kRouteWaves - 1) / kRouteWaves)), block(kRouteWaves * kWave);
    if (p.logits_bf16)
        hipLaunchKernelGGL((moe_route_scored_kernel<NPL, true>), grid, block, 0, s, p);
    else
        hipLaunchKernelGGL((moe_route_scored_kernel<NPL, false>), grid, block, 0, s, p);
    return hipGetLastError();
}

template <int NPL>
hipError_t launch_many(const RouteArgs& p, hipStream_t s)
{
    constexpr int per = kRouteWaves * 4;
    const dim3 grid((unsigned)((p.B + per - 1) / per)), block(kRouteWaves * kWave);
    if (p.logits_bf16)
        hipLaunchKernelGGL((moe_route_scored_many_kernel<NPL, true>), grid, block, 0, s, p);
    else
        hipLaunchKernelGGL((moe_route_scored_many_kernel<NPL, false>), grid, block, 0, s, p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_route_scored(const RouteArgs& p, hipStream_t s)
{
    // us with a wavefront a token and with 16 lanes:
    //   tokens                              1024         2048         4096        16384
    //   8 of 256 experts, 4 of 8 groups   5.6   6.3    6.2   6.4    8.4   6.5    22.4  14.3
    //   8 of 256                          4.7   5.6    5.3   5.7    7.0   5.8    18.5  13.1
    //   2 of 256                          3.5   5.4    3.9   5.5    4.9   5.7    12.2  12.8    two rounds only
    //   8 of 128                          4.3   4.2    4.7   4.3    5.8   4.4    14.0   8.8
    //   8 of 64                           4.0   3.8    4.1   3.8    4.9   3.9    10.7   6.5
    // What goes to the first kernel however many tokens: 8 of 384 experts 7.0, 10.2 and 27.4 us for 2048, 4096 and 16384,
    // 10 of 512 7.3, 10.9 and 29.1, 12 of 256 6.1, 8.2 and 21.5.
    if (p.B >= 2048 && p.k <= kManyK && p.E <= 256 && p.n_group <= 16) {
        if (p.E <= 64)
            return launch_many<4>(p, s);
        if (p.E <= 128)
            return launch_many<8>(p, s);
        return launch_many<16>(p, s);
    }
    const int per_lane = (p.E + kWave - 1) / kWave;
    if (per_lane <= 1) return launch_wave<1>(p, s);
    if (per_lane <= 2) return launch_wave<2>(p, s);
    if (per_lane <= 4) return launch_wave<4>(p, s);
    if (per_lane <= 8) return launch_wave<8>(p, s);
    if (per_lane <= 16) return launch_wave<16>(p, s);
    if (per_lane <= 32) return launch_wave<32>(p, s);
    return hipErrorInvalidValue;
}

}  // namespace moed
