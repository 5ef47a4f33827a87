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
// to be chosen. Round j takes the largest key of the token's lanes (DPP), the lowest lane that holds it writes the
// expert to the token's list in LDS and clears its key. Group values are computed by one lane a group from the keys in
// LDS.
#include "block.h"
#include "mx_device.h"

namespace moed {

namespace {

constexpr int kRouteWaves = 4;

__device__ __forceinline__ uint32_t choice_key(float c)
{
    if (!(c > -__builtin_inff()))
        return 0u;                                // NaN or -infinity
    const uint32_t u = c == 0.0f ? 0u : __float_as_uint(c);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ float choice_of(uint32_t key)
{
    return __uint_as_float((key & 0x80000000u) ? (key & 0x7FFFFFFFu) : ~key);
}

template <int CTRL>
__device__ __forceinline__ uint32_t max_dpp32(uint32_t v)
{
    const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
    return o > v ? o : v;
}

// Largest v of the L lanes of a token, in each of them.
template <int L>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v)
{
    v = max_dpp32<0xB1>(v);                       // quad_perm [1,0,3,2]
    v = max_dpp32<0x4E>(v);                       // quad_perm [2,3,0,1]
    v = max_dpp32<0x141>(v);                      // row_half_mirror
    v = max_dpp32<0x140>(v);                      // row_mirror
    if constexpr (L == 64) {
        const uint32_t o = (uint32_t)__builtin_amdgcn_ds_swizzle((int)v, (0x10 << 10) | 0x1F);
        v = o > v ? o : v;
        const uint32_t a = (uint32_t)__builtin_amdgcn_readlane((int)v, 0);
        const uint32_t c = (uint32_t)__builtin_amdgcn_readlane((int)v, 32);
        v = a > c ? a : c;
    }
    return v;
}

template <int L>
__device__ __forceinline__ double lanes_sum(double v)
{
#pragma unroll
    for (int d = 1; d < L; d <<= 1)
        v += __shfl_xor(v, d);
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

__device__ __forceinline__ void lds_fence()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

}  // namespace

template <int L, int NPL, bool BF16>
__global__ void __launch_bounds__(kRouteWaves * kWave)
moe_route_scored_kernel(RouteArgs p)
{
    constexpr int TW = kWave / L;                 // tokens of a wavefront
    __shared__ uint32_t keys[kRouteWaves * TW][L * NPL];
    __shared__ float scores[kRouteWaves * TW][L * NPL];
    __shared__ int picks[kRouteWaves * TW][kRouteMaxK];
    const int lane = threadIdx.x % kWave, tl = lane % L;
    const int slot = threadIdx.x / L;             // of this token in the workgroup
    const long long first = ((long long)blockIdx.x * kRouteWaves + threadIdx.x / kWave) * TW;
    if (first >= p.B)
        return;                                   // whole wavefronts; no barrier follows
    const long long want = first + lane / L;
    const bool live = want < p.B;                 // the last wavefront's other tokens repeat the last one
    const size_t b = (size_t)(live ? want : p.B - 1);
    const float nan = __builtin_nanf("");
    float l[NPL];
#pragma unroll
    for (int t = 0; t < NPL; ++t) {
        const int e = tl * NPL + t;
        l[t] = nan;
        if (e < p.E)
            l[t] = BF16 ? __uint_as_float((uint32_t) static_cast<const uint16_t*>(p.logits)[b * p.E + e] << 16)
                        : static_cast<const float*>(p.logits)[b * p.E + e];
    }
    float s[NPL];
    if (p.sigmoid) {
#pragma unroll
        for (int t = 0; t < NPL; ++t)
            s[t] = (float)(1.0 / (1.0 + exp(-(double)l[t])));
    } else {
        float m = -__builtin_inff();
#pragma unroll
        for (int t = 0; t < NPL; ++t)
            m = l[t] > m ? l[t] : m;
#pragma unroll
        for (int d = 1; d < L; d <<= 1) {
            const float o = __shfl_xor(m, d);
            m = o > m ? o : m;
        }
        double ex[NPL], sum = 0.0;
#pragma unroll
        for (int t = 0; t < NPL; ++t) {
            ex[t] = l[t] != l[t] ? 0.0 : l[t] == m ? 1.0 : exp((double)l[t] - (double)m);
            sum += ex[t];
        }
        sum = lanes_sum<L>(sum);
#pragma unroll
        for (int t = 0; t < NPL; ++t)
            s[t] = (float)(ex[t] / sum);
    }
    uint32_t key[NPL];
#pragma unroll
    for (int t = 0; t < NPL; ++t) {
        const int e = tl * NPL + t;
        const float c = p.bias && e < p.E ? s[t] + p.bias[e] : s[t];
        key[t] = l[t] != l[t] ? 0u : choice_key(c);
        scores[slot][e] = s[t];
    }
    if (p.topk_group < p.n_group) {
        const int size = p.E / p.n_group;
#pragma unroll
        for (int t = 0; t < NPL; ++t)
            keys[slot][tl * NPL + t] = key[t];
        lds_fence();
        uint32_t worth = 0;                       // of group tl
        if (tl < p.n_group) {
            uint32_t k1 = 0, k2 = 0;
            int at = tl % size;                   // lanes begin at different banks
            for (int i = 0; i < size; ++i) {
                const uint32_t v = keys[slot][tl * size + at];
                at = at + 1 == size ? 0 : at + 1;
                k2 = v > k1 ? k1 : v > k2 ? v : k2;
                k1 = v > k1 ? v : k1;
            }
            worth = k1;
            if (p.top2 && k2 != 0u) {
                // an overflow to -infinity stays above "none"
                const uint32_t sum = choice_key(choice_of(k1) + choice_of(k2));
                worth = sum ? sum : 1u;
            }
        }
        unsigned long long taken = 0;
        for (int j = 0; j < p.topk_group; ++j) {
            const uint32_t m = lanes_max<L>(worth);
            const int win = first_lane<L>(__ballot(worth == m && m != 0u), lane);
            if (win >= 0)
                taken |= 1ull << win;
            if (tl == win)
                worth = 0;
        }
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
    uint32_t best = 0;
#pragma unroll
    for (int t = 0; t < NPL; ++t)
        best = key[t] > best ? key[t] : best;
    int chosen = 0;                               // of this token
    for (int j = 0; j < p.k; ++j) {
        const uint32_t m = lanes_max<L>(best);
        const int win = first_lane<L>(__ballot(best == m && m != 0u), lane);
        chosen += win >= 0;
        if (tl == win) {
            int at = 0;
            best = 0;
#pragma unroll
            for (int t = NPL - 1; t >= 0; --t)
                at = key[t] == m ? t : at;
#pragma unroll
            for (int t = 0; t < NPL; ++t) {
                key[t] = t == at ? 0u : key[t];
                best = key[t] > best ? key[t] : best;
            }
            picks[slot][j] = tl * NPL + at;
        }
    }
    lds_fence();
    double sum = 0.0;
    for (int j = tl; j < chosen; j += L)
        sum += (double)scores[slot][picks[slot][j]];
    if (p.renormalize)
        sum = lanes_sum<L>(sum) + 1e-20;
    else
        sum = 1.0;
    if (!live)
        return;
    const size_t kt = (size_t)p.k + (size_t)p.n_shared;
    for (int j = tl; j < p.k; j += L) {
        const bool ok = j < chosen;
        const int e = ok ? picks[slot][j] : -1;
        p.ids[b * kt + j] = e;
        p.w[b * kt + j] = ok ? (float)((double)scores[slot][ok ? e : 0] / sum * (double)p.routed_scale) : nan;
    }
    for (int i = tl; i < p.n_shared; i += L) {
        p.ids[b * kt + p.k + i] = p.E + i;
        p.w[b * kt + p.k + i] = 1.0f;
    }
}

namespace {

template <int L, int NPL>
hipError_t launch_lanes(const RouteArgs& p, hipStream_t s)
{
    constexpr int per = kRouteWaves * (kWave / L);
    const dim3 grid((unsigned)((p.B + per - 1) / per)), block(kRouteWaves * kWave);
    if (p.logits_bf16)
        hipLaunchKernelGGL((moe_route_scored_kernel<L, NPL, true>), grid, block, 0, s, p);
    else
        hipLaunchKernelGGL((moe_route_scored_kernel<L, NPL, false>), grid, block, 0, s, p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_route_scored(const RouteArgs& p, hipStream_t s)
{
    const int per_lane = (p.E + kWave - 1) / kWave;
    if (per_lane <= 1) return launch_lanes<64, 1>(p, s);
    if (per_lane <= 2) return launch_lanes<64, 2>(p, s);
    if (per_lane <= 4) return launch_lanes<64, 4>(p, s);
    if (per_lane <= 8) return launch_lanes<64, 8>(p, s);
    if (per_lane <= 16) return launch_lanes<64, 16>(p, s);
    if (per_lane <= 32) return launch_lanes<64, 32>(p, s);
    return hipErrorInvalidValue;
}

}  // namespace moed
