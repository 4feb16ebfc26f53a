// attn_shared.h -- where the two halves of a shared-prefix attention meet.
//
// Sequences that begin alike are attended to in two halves: the shared positions by tiles of a group's rows
// (PREFIX), those behind them by sequence (SUFFIX), side by side in one launch.  Each leaves the mean, exponent
// and sum of its columns in the workspace, and the workgroup that is the last to arrive at a sequence's KV head
// (its tiles of either half) joins them and writes o.  All of it passes by agent-scope accesses, as the parts of
// a split do.
#pragma once

#include "attn_common.h"

namespace qg {

// The group of sequence b, which is within the groups: its first sequence.  All lanes of the wave call it.
__device__ __forceinline__ int group_first(const AttnArgs &a, int b)
{
    const int lane = threadIdx.x & 63;
    int first = 0;
    for (int g0 = 0; g0 < a.n_group; g0 += 64) {
        const int f = g0 + lane < a.n_group ? max(a.group_start[g0 + lane], 0) : 0x7fffffff;
        const uint64_t below = __ballot(f <= b);
        if (!below)
            break;
        first = __builtin_amdgcn_readlane(f, 63 - __builtin_clzll(below));
    }
    return first;
}

// Tiles of 16 columns that hold columns of row m of a group, and those of its own positions.
__device__ __forceinline__ int meeting(int m, int group)
{
    return ((m + 1) * group - 1) / 16 - m * group / 16 + 1 + (group + 15) / 16;
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t meet_means(const AttnArgs &a, int half)
{
    const int64_t n = (int64_t)a.rows_in_all * a.nq * a.c.hd;
    return __builtin_amdgcn_make_buffer_rsrc(a.means + half * n, 0, (int)(n * 4), 0x00020000);
}
__device__ __forceinline__ __amdgpu_buffer_rsrc_t meet_stats(const AttnArgs &a, int half)
{
    const int64_t n = (int64_t)a.rows_in_all * a.nq * 2;
    return __builtin_amdgcn_make_buffer_rsrc(a.stats + half * n, 0, (int)(n * 4), 0x00020000);
}

// One half's four channels d4 of row and head `at`.
template <int D>
__device__ __forceinline__ void meet_put(const AttnArgs &a, int half, int64_t at, int d4, af4 mean, float m, float l)
{
    put4(meet_means(a, half), (uint32_t)(at * D + 4 * d4), mean);
    if (d4 == 0)
        put2(meet_stats(a, half), (uint32_t)(2 * at), m, l);
}

// A workgroup's columns are those of rows row0 + [0, n) of a KV head (n <= 16; members(i) arrivals at row i, 0:
// it does not meet).  Joins the rows of which it is the last to arrive.
template <int D, class Members>
__device__ __forceinline__ void meet(const AttnArgs &a, int row0, int n, int hkv, int *done, Members members)
{
    const int tid = threadIdx.x;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (tid < n) {
        const int all = members(tid);
        unsigned int *cnt = a.meet + (int64_t)(row0 + tid) * a.c.nkv + hkv;
        int last = 0;
        if (all > 0 && __hip_atomic_fetch_add(cnt, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + 1 ==
                           (unsigned int)all) {
            last = 1;
            __hip_atomic_store(cnt, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        done[tid] = last;
    }
    __syncthreads();
    asm volatile("" ::: "memory");
    const int items = a.group * (D / 4);
    for (int i = 0; i < n; ++i) {
        if (!done[i])
            continue;
        for (int e = tid; e < items; e += 256) {
            const int d4 = e % (D / 4);
            const int64_t at = (int64_t)(row0 + i) * a.nq + hkv * a.group + e / (D / 4);
            float m[2], l[2];
            af4 x[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                get2(meet_stats(a, h), (uint32_t)(2 * at), m[h], l[h]);
                x[h] = get4(meet_means(a, h), (uint32_t)(at * D + 4 * d4));
            }
            *reinterpret_cast<af4 *>(a.o + at * D + 4 * d4) = join_means(x[0], m[0], l[0], x[1], m[1], l[1]);
        }
    }
}

}  // namespace qg
