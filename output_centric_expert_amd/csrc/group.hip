// Routed slots sorted by expert: for ids[t], t = b*k + j, the stable counting
// sort order (slots of expert 0 first, each expert's in increasing t), every
// slot's place in it, and where each expert's slots begin.
//
// Slots are taken in blocks of 16 wavefronts; a wavefront owns PER*64
// consecutive slots and takes them 64 at a time. Lanes with the same id are
// found with one ballot per id bit, so a slot's rank among its wavefront's
// earlier slots of the expert is a count in LDS plus a popcount: no atomics,
// no dependence on the order in which wavefronts run. Counts of wavefronts
// (and, past one block, of blocks) are then summed in slot order.
//
// One block covers n <= 8192 slots in one launch (64 tokens of 8 of 256
// experts: 3.6 us, its barriers and round trips). Larger lists take two
// launches: the blocks' counts to the workspace, then every block adds up the
// counts itself (blocks*E words out of L2, all threads at once where E <= 512:
// 16384 tokens of 8 of 128 experts take 8.8 us, 20.8 us with one thread an
// expert). Past kGroupScan blocks a launch in between scans the counts, so that
// the time grows with the slots.
#include "mx_device.h"
#include "prompt.h"

namespace moed {

namespace {

constexpr int kGroupThreads = 1024;
constexpr int kGroupWavesN = kGroupThreads / kWave;
// Past this many blocks their counts are scanned in a launch of its own. Adding them up in every block grows with the
// square of their number: 2^24 slots, 2048 blocks, take 447 us with 128 experts and 1780 with 2048 that way, 160 and 248
// with the scan; at 256 blocks (2^21 slots) both take about the same (8 experts 18.7 and 19.9, 128 experts 28.8 and
// 28.4, 2048 experts 66 and 45), and below the scan's launch is the larger part (2^17 slots of 128 experts 9.6 and 12.2).
constexpr int kGroupScan = 256;

// Lanes of the wavefront that hold the same id (ids < 2^bits), among `live`.
__device__ __forceinline__ unsigned long long same_id(int id, int bits, unsigned long long live)
{
    unsigned long long m = live;
    for (int i = 0; i < bits; ++i) {
        const unsigned long long b = __ballot((id >> i) & 1);
        m &= ((id >> i) & 1) ? b : ~b;
    }
    return m;
}

// Adds expert e's counts of blocks from .. to-1 (`earlier`: of those before blk).
__device__ __forceinline__ void add_counts(const int32_t* counts, int e, int E, int from, int to, int blk, int& earlier,
                                           int& all)
{
#pragma unroll 8
    for (int q = from; q < to; ++q) {
        const int c = counts[(size_t)q * E + e];
        earlier += q < blk ? c : 0;
        all += c;
    }
}

// Sum of v over the threads before this one, and over all (block of 1024).
__device__ __forceinline__ int block_exclusive(int v, int* wsum, int& total)
{
    const int lane = threadIdx.x % kWave, w = threadIdx.x / kWave;
    int inc = v;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const int o = __shfl_up(inc, d);
        if (lane >= d)
            inc += o;
    }
    if (lane == kWave - 1)
        wsum[w] = inc;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int q = 0; q < kGroupWavesN; ++q) {
        const int c = wsum[q];
        before += q < w ? c : 0;
        all += c;
    }
    __syncthreads();
    total = all;
    return before + inc - v;
}

}  // namespace

// Counts of one block's slots per expert, to the workspace: counts[block][E].
template <int PER>
__global__ void __launch_bounds__(kGroupThreads)
moe_group_count_kernel(const int32_t* ids, int n, int E, int32_t* counts)
{
    extern __shared__ int hist[];
    for (int e = threadIdx.x; e < E; e += kGroupThreads)
        hist[e] = 0;
    __syncthreads();
    const long long base = (long long)blockIdx.x * (PER * kGroupThreads);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const long long t = base + i * kGroupThreads + threadIdx.x;
        const int id = t < n ? ids[t] : -1;
        if ((unsigned)id < (unsigned)E)
            atomicAdd(&hist[id], 1);              // integers: any order gives the same counts
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kGroupThreads)
        counts[(size_t)blockIdx.x * E + e] = hist[e];
}

// counts[block][E] -> slots of the blocks before each (in place), and all blocks' sum in row nblk. A workgroup takes up
// to 64 experts; its threads share the blocks in `parts` runs, whose sums meet in LDS.
__global__ void __launch_bounds__(kGroupThreads)
moe_group_scan_kernel(int32_t* counts, int E, int nblk)
{
    __shared__ int sums[kGroupThreads];
    const int columns = E < kWave ? E : kWave, parts = kGroupThreads / columns;
    const int q = threadIdx.x / columns, c = threadIdx.x % columns, e = blockIdx.x * columns + c;
    const int per = (nblk + parts - 1) / parts;
    const int from = q * per < nblk ? q * per : nblk, to = from + per < nblk ? from + per : nblk;
    const bool live = q < parts && e < E;
    int sum = 0;
    if (live)
#pragma unroll 8
        for (int b = from; b < to; ++b)
            sum += counts[(size_t)b * E + e];
    sums[threadIdx.x] = sum;
    __syncthreads();
    if (!live)
        return;                                   // no barrier follows
    int at = 0;
    for (int i = 0; i < q; ++i)
        at += sums[i * columns + c];
    if (q == parts - 1)
        counts[(size_t)nblk * E + e] = at + sum;
#pragma unroll 8
    for (int b = from; b < to; ++b) {
        const int n = counts[(size_t)b * E + e];
        counts[(size_t)b * E + e] = at;
        at += n;
    }
}

// nblk = 1: counts unused. scanned: counts are those of the scan. LDS: E ints (starts), then 16*E uint16 (per-wavefront
// counts).
template <int PER>
__global__ void __launch_bounds__(kGroupThreads)
moe_group_place_kernel(const int32_t* ids, int n, int E, int bits, int nblk, bool scanned, const int32_t* counts,
                       int32_t* order, int32_t* position, int32_t* offsets)
{
    extern __shared__ int start[];                // E: first place of this block's slots of each expert
    uint16_t* cnt = reinterpret_cast<uint16_t*>(start + E);    // [16][E]
    __shared__ int wsum[kGroupWavesN];
    __shared__ int sums[2 * kGroupThreads];
    const int tid = threadIdx.x, lane = tid % kWave, w = tid / kWave;
    const int blk = blockIdx.x;
    const long long first = (long long)blk * (PER * kGroupThreads) + (long long)w * (PER * kWave) + lane;
    int id[PER], rank[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const long long t = first + i * kWave;
        id[i] = t < n ? ids[t] : -1;
    }
    for (int i = tid; i < (kGroupWavesN * E + 1) / 2; i += kGroupThreads)
        reinterpret_cast<uint32_t*>(cnt)[i] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const bool ok = (unsigned)id[i] < (unsigned)E;
        const unsigned long long live = __ballot(ok);
        const unsigned long long m = same_id(ok ? id[i] : 0, bits, live);
        rank[i] = 0;
        if (ok) {
            const int before = __popcll(m & ((1ull << lane) - 1ull));
            const int have = cnt[w * E + id[i]];
            rank[i] = have + before;
            // one lane per id writes, after every lane of the wavefront has read
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            if (before == 0)
                cnt[w * E + id[i]] = (uint16_t)(have + __popcll(m));
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    __syncthreads();
    // few experts: the blocks' counts are added by parts = 1024 / E threads an expert
    const int parts = nblk > 1 && !scanned && E < kGroupThreads ? kGroupThreads / E : 1;
    if (parts > 1) {
        const int q = tid / E, e = tid - q * E;
        if (q < parts) {
            int earlier = 0, all = 0;
            const int per = (nblk + parts - 1) / parts;
            add_counts(counts, e, E, q * per, q * per + per < nblk ? q * per + per : nblk, blk, earlier, all);
            sums[(2 * q) * E + e] = earlier;
            sums[(2 * q + 1) * E + e] = all;
        }
        __syncthreads();
    }
    // per expert: earlier wavefronts of this block, earlier blocks, all blocks
    int done = 0;                                 // slots of the experts before this chunk of 1024 experts
    for (int e0 = 0; e0 < E; e0 += kGroupThreads) {
        const int e = e0 + tid;
        int mine = 0, earlier = 0, all = 0;
        if (e < E) {
#pragma unroll
            for (int q = 0; q < kGroupWavesN; ++q) {
                const int c = cnt[q * E + e];
                cnt[q * E + e] = (uint16_t)mine;
                mine += c;
            }
            if (nblk == 1) {
                all = mine;
            } else if (scanned) {
                earlier = counts[(size_t)blk * E + e];
                all = counts[(size_t)nblk * E + e];
            } else if (parts == 1) {
                add_counts(counts, e, E, 0, nblk, blk, earlier, all);
            } else {                              // E <= 512: summed above by all threads
                for (int q = 0; q < parts; ++q) {
                    earlier += sums[(2 * q) * E + e];
                    all += sums[(2 * q + 1) * E + e];
                }
            }
        }
        int total = 0;
        const int at = done + block_exclusive(all, wsum, total);
        if (e < E) {
            start[e] = at + earlier;
            if (blk == 0)
                offsets[e] = at;
        }
        done += total;
    }
    if (blk == 0 && tid == 0)
        offsets[E] = done;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const long long t = first + i * kWave;
        if (t >= n)
            continue;
        int at = -1;
        if ((unsigned)id[i] < (unsigned)E) {
            at = start[id[i]] + cnt[w * E + id[i]] + rank[i];
            order[at] = (int32_t)t;
        }
        position[t] = at;
        if (t >= done)
            order[t] = -1;                        // places behind the last expert's slots
    }
}

size_t group_workspace(int n, int E)
{
    if (n <= kGroupOneBlock)
        return 0;
    const size_t per = n <= (1 << 18) ? 2 : 8, nblk = ((size_t)n + per * kGroupThreads - 1) / (per * kGroupThreads);
    return (nblk + (nblk > kGroupScan ? 1 : 0)) * (size_t)E * 4u;
}

template <int PER>
static hipError_t launch_place(const int32_t* ids, int n, int E, int nblk, int32_t* counts, int32_t* order,
                               int32_t* position, int32_t* offsets, hipStream_t s)
{
    int bits = 0;
    while ((1 << bits) < E)
        ++bits;
    const size_t lds = (size_t)E * 4 + ((size_t)kGroupWavesN * E + 1) / 2 * 4;
    const void* f = reinterpret_cast<const void*>(&moe_group_place_kernel<PER>);
    if (lds > 49152)                              // beside the kernel's own arrays
        if (hipError_t e = set_max_dynamic_lds(f, (int)lds))
            return e;
    if (nblk > 1) {
        hipLaunchKernelGGL((moe_group_count_kernel<PER>), dim3((unsigned)nblk), dim3(kGroupThreads), (size_t)E * 4, s, ids,
                           n, E, counts);
        if (hipError_t e = hipGetLastError())
            return e;
    }
    const bool scanned = nblk > kGroupScan;
    if (scanned) {
        hipLaunchKernelGGL(moe_group_scan_kernel, dim3((unsigned)(E + kWave - 1) / kWave), dim3(kGroupThreads), 0, s, counts,
                           E, nblk);
        if (hipError_t e = hipGetLastError())
            return e;
    }
    hipLaunchKernelGGL((moe_group_place_kernel<PER>), dim3((unsigned)nblk), dim3(kGroupThreads), lds, s, ids, n, E, bits,
                       nblk, scanned, counts, order, position, offsets);
    return hipGetLastError();
}

hipError_t launch_group(const int32_t* ids, int n, int E, int32_t* counts, int32_t* order, int32_t* position,
                        int32_t* offsets, hipStream_t s)
{
    if (n <= kGroupThreads)
        return launch_place<1>(ids, n, E, 1, counts, order, position, offsets, s);
    if (n <= kGroupOneBlock)
        return launch_place<8>(ids, n, E, 1, counts, order, position, offsets, s);
    if (n <= (1 << 18))
        return launch_place<2>(ids, n, E, (n + 2 * kGroupThreads - 1) / (2 * kGroupThreads), counts, order, position,
                               offsets, s);
    return launch_place<8>(ids, n, E, (int)(((long long)n + 8 * kGroupThreads - 1) / (8 * kGroupThreads)), counts, order,
                           position, offsets, s);
}

}  // namespace moed
