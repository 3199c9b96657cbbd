// sort.hip -- a router's choices in order of experts: a stable counting sort.
//
//   offsets[e]   number of slots whose expert is below e
//   position[s]  offsets[e] + number of slots before s with the same expert e
//   order        the inverse: order[position[s]] = s
//
// Slots outside [0, experts) get position -1; order past offsets[experts] is
// -1.  A wave takes 64 consecutive slots at a time; which of its lanes hold the
// same expert follows from one ballot for each bit of the expert's number, so
// that ranks come without atomics and in the order of slots.  Each wave counts
// in its own row of LDS, a scan over waves and experts turns the counts into
// first places, and a second walk over the same slots hands them out.
//
// Few slots: one workgroup.  More: a first launch counts for each workgroup's
// slots, in the second each workgroup sums the counts before its own.  Bound by
// latency, loads, ballots and scans one after the other (one MI355X: 64 x 8
// choices of 256 experts 3.9 us, 32769 x 8 of 128 3.3 + 8.8 us, for 3 MB).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "experts.hpp"

namespace qgemm {

namespace {

constexpr int THREADS = 1024, WAVES = THREADS / 64;
constexpr int ONE_WORKGROUP = 8192;    // slots that one workgroup sorts alone
constexpr int MOST_BLOCKS = 256;
constexpr int KEEP = 4;                // slots of a lane kept in registers

// The lanes of the wave whose e equals this lane's, among the live ones.
__device__ __forceinline__ uint64_t same_lanes(int e, bool live, int bits)
{
    uint64_t m = __ballot(live);
    for (int b = 0; b < bits; ++b) {
        const uint64_t v = __ballot((e >> b) & 1);
        m &= (e >> b) & 1 ? v : ~v;
    }
    return m;
}

// The sum over this lane and those below it.
__device__ __forceinline__ int scan_lanes(int v, int lane)
{
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int u = __shfl_up(v, off);
        v += lane >= off ? u : 0;
    }
    return v;
}

__global__ void __launch_bounds__(THREADS) moe_count_kernel(SortArgs a)
{
    __shared__ int hist[MOE_MAX_EXPERTS];
    const int t = threadIdx.x;
    for (int e = t; e < a.experts; e += THREADS)
        hist[e] = 0;
    __syncthreads();
    const int lo = blockIdx.x * a.chunk, hi = min(a.slots, lo + a.chunk);
    for (int s = lo + t; s < hi; s += THREADS) {
        const int e = a.ids[s];
        if ((unsigned)e < (unsigned)a.experts)
            atomicAdd(&hist[e], 1);
    }
    __syncthreads();
    for (int e = t; e < a.experts; e += THREADS)
        a.hist[blockIdx.x * a.experts + e] = hist[e];
}

template <bool MANY>
__global__ void __launch_bounds__(THREADS) moe_sort_kernel(SortArgs a)
{
    __shared__ int place[WAVES * MOE_MAX_EXPERTS];   // [WAVES][experts]: counts, then next places
    __shared__ int wave_sum[WAVES];
    __shared__ int before[MANY ? MOE_MAX_EXPERTS : 1], total[MANY ? MOE_MAX_EXPERTS : 1];
    const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int E = a.experts;
    const int bits = 32 - __builtin_clz(max(E - 1, 1));
    // this wave's slots, and the experts of the first of them (a wave seldom has
    // more), loaded before anything else
    const int first = MANY ? blockIdx.x * a.chunk : 0, last = MANY ? min(a.slots, first + a.chunk) : a.slots;
    const int per = ((last - first + WAVES - 1) / WAVES + 63) / 64 * 64;
    const int lo = min(first + wave * per, last), hi = min(lo + per, last);
    int ids[KEEP];
    auto load = [&](int s0) {
#pragma unroll
        for (int i = 0; i < KEEP; ++i) {
            const int s = s0 + 64 * i + lane;
            ids[i] = s < hi ? a.ids[s] : -1;
        }
    };
    load(lo);
    for (int i = t; i < WAVES * E; i += THREADS)
        place[i] = 0;
    if constexpr (MANY) {
        // counts of the workgroups before this one, and of all: THREADS / E (at
        // least one) threads share an expert
        for (int e = t; e < E; e += THREADS)
            before[e] = total[e] = 0;
        __syncthreads();
        const int parts = max(THREADS / E, 1);
        for (int i = t; i < parts * E; i += THREADS) {
            const int e = i % E, part = i / E;
            int b4 = 0, all = 0;
            for (int b0 = part; b0 < a.blocks; b0 += 8 * parts) {   // eight counts in flight
                int n[8];
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    n[u] = b0 + u * parts < a.blocks ? a.hist[(b0 + u * parts) * E + e] : 0;
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    all += n[u];
                    b4 += b0 + u * parts < (int)blockIdx.x ? n[u] : 0;
                }
            }
            atomicAdd(&before[e], b4);
            atomicAdd(&total[e], all);
        }
    }
    __syncthreads();

    int *mine = place + wave * E;
    for (int s0 = lo; s0 < hi; s0 += 64 * KEEP) {
        if (s0 > lo)
            load(s0);
#pragma unroll
        for (int i = 0; i < KEEP; ++i) {
            if (s0 + 64 * i >= hi)
                break;
            const int e = ids[i];
            const bool live = (unsigned)e < (unsigned)E;
            const uint64_t m = same_lanes(e, live, bits);
            if (live && (m & ((1ull << lane) - 1)) == 0)
                mine[e] += __popcll(m);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");   // the next slots' lanes read it
        }
    }
    __syncthreads();

    // first places: over the waves of each expert, then over the experts
    // (thread t has expert t: experts <= THREADS)
    int count[WAVES], n = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w)
        count[w] = t < E ? place[w * E + t] : 0;
    if constexpr (MANY) {
        n = t < E ? total[t] : 0;
    } else {
#pragma unroll
        for (int w = 0; w < WAVES; ++w)
            n += count[w];
    }
    const int scan = scan_lanes(n, lane);
    if (lane == 63)
        wave_sum[wave] = scan;
    __syncthreads();
    const int waves_scan = scan_lanes(lane < WAVES ? wave_sum[lane] : 0, lane);
    const int live_rows = __builtin_amdgcn_readlane(waves_scan, WAVES - 1);
    const int at = scan - n + (wave ? __builtin_amdgcn_readlane(waves_scan, wave - 1) : 0);
    if (t < E) {
        int base = at;
        if constexpr (MANY)
            base += before[t];
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            place[w * E + t] = base;
            base += count[w];
        }
        if (!MANY || blockIdx.x == 0) {
            a.offsets[t] = at;
            if (t == 0)
                a.offsets[E] = live_rows;
        }
    }
    __syncthreads();

    for (int s0 = lo; s0 < hi; s0 += 64 * KEEP) {
        if (hi - lo > 64 * KEEP)
            load(s0);
#pragma unroll
        for (int i = 0; i < KEEP; ++i) {
            if (s0 + 64 * i >= hi)
                break;
            const int s = s0 + 64 * i + lane, e = ids[i];
            const bool live = (unsigned)e < (unsigned)E;
            const uint64_t m = same_lanes(e, live, bits), lower = m & ((1ull << lane) - 1);
            int p = -1;
            if (live)
                p = mine[e] + __popcll(lower);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");   // every lane has read its place
            if (live && lower == 0)
                mine[e] += __popcll(m);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            if (s < hi)
                a.position[s] = p;
            if (live)
                a.order[p] = s;
        }
    }
    // places that no slot takes
    for (int r = max(live_rows, first) + t; r < last; r += THREADS)
        a.order[r] = -1;
}

}  // namespace

int64_t sort_plan(SortArgs &a)
{
    if (a.slots <= ONE_WORKGROUP) {
        a.blocks = 1;
        a.chunk = a.slots;
        return 0;
    }
    a.chunk = std::max(2048, (int)(((int64_t)a.slots + MOST_BLOCKS - 1) / MOST_BLOCKS));
    a.blocks = (a.slots + a.chunk - 1) / a.chunk;
    return (int64_t)a.blocks * a.experts * 4;
}

hipError_t launch_moe_sort(const SortArgs &a, hipStream_t s)
{
    if (a.blocks == 1) {
        hipLaunchKernelGGL((moe_sort_kernel<false>), dim3(1), dim3(THREADS), 0, s, a);
        return hipGetLastError();
    }
    hipLaunchKernelGGL(moe_count_kernel, dim3(a.blocks), dim3(THREADS), 0, s, a);
    if (const hipError_t e = hipGetLastError())
        return e;
    hipLaunchKernelGGL((moe_sort_kernel<true>), dim3(a.blocks), dim3(THREADS), 0, s, a);
    return hipGetLastError();
}

}  // namespace qgemm
