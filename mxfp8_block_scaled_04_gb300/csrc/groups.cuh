// Per-expert row offsets in shared memory: checked, with the tiles of the groups before each one.
#pragma once

#include <cstdint>

namespace mxfp8 {

constexpr int kGroupMax = 512;

template <bool USED>
struct GroupTable {
    int64_t offset[kGroupMax + 1];
    int tile[kGroupMax + 1];   // tiles (of the kernel's rows) before group g
    int plane[kGroupMax + 1];  // 128-row tiles of scale plane before group g
    unsigned long long scan[32];

    // The group of row tile t: tile[g] <= t < tile[g + 1].
    __device__ __forceinline__ int find(int t, int num_groups) const
    {
        int lo = 0, hi = num_groups;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (tile[mid] <= t)
                lo = mid;
            else
                hi = mid;
        }
        return lo;
    }
};
template <>
struct GroupTable<false> {};

// An offset in rows of the operand; one that is out of range (and would overflow) stays out of range.
template <int TIMES>
__device__ __forceinline__ int64_t scaled_offset(int64_t offset, int64_t total)
{
    if constexpr (TIMES == 1)
        return offset;
    else
        return offset < 0 ? -1 : offset > total ? total + 1 : offset * TIMES;
}

// Load and check the offsets (from 0, non-decreasing, none past total; rows past the last one belong to no group); all
// threads of the CTA.  Returns the number of row tiles of ROWS rows over all groups, or -1 for bad offsets.  Both
// prefixes come from one scan of a packed count (the low half stays below 2^32: at most total / 128 + groups).  Offsets and
// total count rows of the operand, TIMES of which stand for one row that the caller counts.
template <int THREADS, int ROWS, int TIMES = 1>
__device__ __forceinline__ int group_setup(GroupTable<true> &g, const int64_t *offsets, int num_groups, int64_t total)
{
    constexpr int kItems = (kGroupMax + THREADS - 1) / THREADS;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int i = tid; i <= num_groups; i += THREADS)
        g.offset[i] = scaled_offset<TIMES>(offsets[i], total);
    __syncthreads();
    int bad = tid == 0 && (g.offset[0] != 0 || g.offset[num_groups] > total);
    for (int i = tid; i < num_groups; i += THREADS)
        bad |= g.offset[i + 1] < g.offset[i];
    if (__syncthreads_or(bad))
        return -1;
    unsigned long long c[kItems], sum = 0;
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
        const int i = tid * kItems + k;
        c[k] = 0;
        if (i < num_groups) {
            const unsigned long long rows = static_cast<unsigned long long>(g.offset[i + 1] - g.offset[i]);
            c[k] = ((rows + ROWS - 1) / ROWS << 32) | ((rows + 127) / 128);
        }
        sum += c[k];
    }
    unsigned long long incl = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const unsigned long long v = __shfl_up_sync(0xFFFFFFFFu, incl, d);
        if (lane >= d)
            incl += v;
    }
    if (lane == 31)
        g.scan[warp] = incl;
    __syncthreads();
    unsigned long long base = 0, all = 0;
    for (int w = 0; w < THREADS / 32; ++w) {
        base += w < warp ? g.scan[w] : 0;
        all += g.scan[w];
    }
    unsigned long long at = base + incl - sum;
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
        const int i = tid * kItems + k;
        if (i < num_groups) {
            g.tile[i] = static_cast<int>(at >> 32);
            g.plane[i] = static_cast<int>(at & 0xFFFFFFFFu);
        }
        at += c[k];
    }
    if (tid == 0) {
        g.tile[num_groups] = static_cast<int>(all >> 32);
        g.plane[num_groups] = static_cast<int>(all & 0xFFFFFFFFu);
    }
    __syncthreads();
    return static_cast<int>(all >> 32);
}

}  // namespace mxfp8
