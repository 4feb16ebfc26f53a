// route_kernels.hip -- routing of rows to experts: scores, groups, top-k, weights.
//
// s = softmax(z) or sigmoid(z) over a row's experts, choice c = s + bias; the topk_group groups
// with the largest sum of their best group_top c stay; the topk largest c among them, ties to the
// lower index; weights s (renormalised) * scale.
//
// One wave per row, lane l holding experts NI l .. NI l + NI - 1, so that the first of several lanes
// with equal choices has the lowest expert and a group is a run of lanes.  Scores and choices are
// f64: two choices that differ by less than an f32 rounding (a bias near the scores' own spacing)
// must come out in their true order, and gfx950 runs f64 at the f32 rate.  A choice is compared as
// the unsigned image of its bits (order-preserving), 0 meaning "not selectable".
//
// The rounds of the selection first compare only the upper 32 bits of the images, with the lane's
// slot in the lowest of them: a round is a maximum over the wave (lane shifts in the VALU) and a
// vote.  Two choices next to each other in the result that share the compared bits (2^-16 of their
// value or nearer) may be in the wrong order; then, for the whole wave, the selection is done anew
// on all 64 bits.
//
// Bound by VALU issue, not by the 8.7 MB it moves: 8000 x 256, sigmoid, 8 groups, top 8 of 4 groups,
// takes 31.1 us with shuffled 64-bit maxima and a serial scan of the groups, 15.2 us with lane shifts
// and 64-bit rounds, 13 us as it is (700 VALU instructions a row); 16 x 64, top 8, 5.4 us, of which the
// kernel is 3.2.  8000 x 1000, softmax, 8 groups of 125 (no run of lanes), a lane scanning a group: 192 us,
// eight lanes 69.
#include <hip/hip_runtime.h>

#include "attn_internal.h"

namespace qg {

// Order-preserving image of a double; NaN counts as -inf; never 0.
__device__ __forceinline__ uint64_t route_key(double c)
{
    if (!(c == c))
        c = -INFINITY;
    const uint64_t b = __builtin_bit_cast(uint64_t, c + 0.0);   // -0 counts as +0
    return b >> 63 ? ~b : b | 0x8000000000000000ull;
}

// Lane shifts of the wave-wide reductions: after the six steps lane 63 has the result; a lane that
// nothing is shifted into takes `none`.
template <int CTRL, int ROWS, class V>
__device__ __forceinline__ V dpp_or(V none, V v)
{
    return __builtin_bit_cast(V, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, none),
                                                             __builtin_bit_cast(int, v), CTRL, ROWS, 0xF, false));
}
template <class V, class F>
__device__ __forceinline__ V wave_reduce(V v, V none, F f)
{
    v = f(v, dpp_or<0x111, 0xF>(none, v));              // row_shr 1, 2, 4, 8
    v = f(v, dpp_or<0x112, 0xF>(none, v));
    v = f(v, dpp_or<0x114, 0xF>(none, v));
    v = f(v, dpp_or<0x118, 0xF>(none, v));
    v = f(v, dpp_or<0x142, 0xA>(none, v));              // row 0 -> 1, 2 -> 3
    v = f(v, dpp_or<0x143, 0xC>(none, v));              // rows 0, 1 -> 2, 3
    return __builtin_bit_cast(V, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v)
{
    return wave_reduce(v, 0u, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_add(double v)
{
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = dpp_or<CTRL, ROWS>(0u, (uint32_t)b), hi = dpp_or<CTRL, ROWS>(0u, (uint32_t)(b >> 32));
    return v + __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double lane_double(double v, int lane)
{
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)b, lane);
    const uint32_t hi = __builtin_amdgcn_readlane((uint32_t)(b >> 32), lane);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double wave_sum(double v)
{
    v = dpp_add<0x111, 0xF>(v);
    v = dpp_add<0x112, 0xF>(v);
    v = dpp_add<0x114, 0xF>(v);
    v = dpp_add<0x118, 0xF>(v);
    v = dpp_add<0x142, 0xA>(v);
    v = dpp_add<0x143, 0xC>(v);
    return lane_double(v, 63);
}

// First lane that holds the wave's largest key.
__device__ __forceinline__ int best_lane(uint64_t key)
{
    const uint32_t hi = (uint32_t)(key >> 32), lo = (uint32_t)key, top = wave_max(hi);
    uint64_t who = __ballot(hi == top);
    if (__popcll(who) > 1) {
        const uint32_t low = wave_max(hi == top ? lo : 0u);
        who = __ballot(hi == top && lo == low);
    }
    return __ffsll((unsigned long long)who) - 1;
}

// The wave's largest key and the lowest index holding it (any layout of the indices).
__device__ __forceinline__ void wave_best(uint64_t &key, int &idx)
{
#pragma unroll
    for (int x = 32; x; x >>= 1) {
        const uint64_t k2 = __shfl_xor((unsigned long long)key, x);
        const int i2 = __shfl_xor(idx, x);
        if (k2 > key || (k2 == key && i2 < idx)) {
            key = k2;
            idx = i2;
        }
    }
}

// Maximum and minimum of values that are no NaN, in one instruction each (fmax would first quieten
// its operands).
__device__ __forceinline__ double max64(double a, double b)
{
    double r;
    asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}
__device__ __forceinline__ double min64(double a, double b)
{
    double r;
    asm("v_min_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}
// Best two of a run of values.
struct Top2 {
    double a, b;
    __device__ __forceinline__ void add(double c)
    {
        b = max64(b, min64(a, c));
        a = max64(a, c);
    }
    __device__ __forceinline__ void merge(double a2, double b2)
    {
        b = max64(min64(a, a2), max64(b, b2));
        a = max64(a, a2);
    }
};

// Eight and sixteen experts a lane are held to 128 registers (sixteen spill 17): left alone, all their
// exponentials run side by side in 478 (8000 x 1024: 84.6 us, 40.2; x 512: 23.7, 21.9).
template <int NI>
__global__ __launch_bounds__(256, NI >= 8 ? 4 : 1) void k_route(RouteArgs a)
{
    __shared__ double s_c[4][64 * NI];
    __shared__ uint8_t s_keep[4][64 * NI];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int64_t r = (int64_t)blockIdx.x * 4 + wave;
    if (r >= a.n_rows)
        return;                                   // no workgroup barrier below
    const float *zr = a.z + r * a.n_exp;
    const int e0 = NI * lane;
    float z[NI];
    double s[NI], c[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i)
        z[i] = e0 + i < a.n_exp ? zr[e0 + i] : -INFINITY;
    if (a.sigmoid) {
#pragma unroll
        for (int i = 0; i < NI; ++i)
            s[i] = 1.0 / (1.0 + exp(-(double)z[i]));
    } else {
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < NI; ++i)
            m = fmaxf(m, z[i]);
        m = wave_reduce(m, -INFINITY, [](float x, float y) { return fmaxf(x, y); });
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            s[i] = e0 + i < a.n_exp ? exp((double)z[i] - (double)m) : 0.0;
            sum += s[i];
        }
        const double inv = 1.0 / wave_sum(sum);
#pragma unroll
        for (int i = 0; i < NI; ++i)
            s[i] *= inv;
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        c[i] = a.bias && e0 + i < a.n_exp ? s[i] + (double)a.bias[e0 + i] : s[i];
        c[i] = c[i] == c[i] ? c[i] : -INFINITY;
    }

    uint32_t keep = ~0u;                          // bit i: expert e0 + i is in a group that stays
    if (a.n_group > 1) {
        if (a.run_log2 >= 0) {
            // a group is a run of 2^k lanes
            Top2 t = {-INFINITY, -INFINITY};
#pragma unroll
            for (int i = 0; i < NI; ++i)
                t.add(c[i]);
            for (int x = 0; x < a.run_log2; ++x)
                t.merge(__shfl_xor(t.a, 1 << x), __shfl_xor(t.b, 1 << x));
            const int g = lane >> a.run_log2;
            uint64_t gk = g < a.n_group ? route_key(a.group_top == 2 ? t.a + t.b : t.a) : 0;
            keep = 0;
            for (int x = 0; x < a.topk_group; ++x)
                if (best_lane(gk) >> a.run_log2 == g) {
                    gk = 0;
                    keep = ~0u;
                }
        } else {
            // any other size: the choices in LDS, 2^k lanes per group, or one for groups lane, lane + 64, ...
            const int size = a.n_exp / a.n_group;
            const int lanes = a.n_group > 32 ? 1 : 1 << (31 - __builtin_clz(64 / a.n_group));
            const int step = 64 / lanes, first = lane / lanes, sub = lane % lanes;
            auto wave_sync = []() {
                __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
                __builtin_amdgcn_wave_barrier();
                __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
            };
#pragma unroll
            for (int i = 0; i < NI; ++i)
                s_c[wave][e0 + i] = c[i];
            wave_sync();
            uint64_t gk[NI];
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int g = first + step * i;
                gk[i] = 0;
                s_keep[wave][lane + 64 * i] = 0;
                if (step * i < a.n_group) {
                    Top2 t = {-INFINITY, -INFINITY};
                    if (g < a.n_group)
                        for (int j = sub; j < size; j += lanes)
                            t.add(s_c[wave][g * size + j]);
                    for (int x = 1; x < lanes; x *= 2)
                        t.merge(__shfl_xor(t.a, x), __shfl_xor(t.b, x));
                    if (g < a.n_group && sub == 0)
                        gk[i] = route_key(a.group_top == 2 ? t.a + t.b : t.a);
                }
            }
            for (int x = 0; x < a.topk_group; ++x) {
                uint64_t k = 0;
                int idx = 0x7fffffff;
#pragma unroll
                for (int i = 0; i < NI; ++i)
                    if (gk[i] > k) {
                        k = gk[i];
                        idx = first + step * i;
                    }
                wave_best(k, idx);
#pragma unroll
                for (int i = 0; i < NI; ++i)
                    if (sub == 0 && idx == first + step * i) {
                        gk[i] = 0;
                        s_keep[wave][idx] = 1;
                    }
            }
            wave_sync();
            keep = 0;
#pragma unroll
            for (int i = 0; i < NI; ++i)
                if (e0 + i < a.n_exp && s_keep[wave][(e0 + i) / size])
                    keep |= 1u << i;
        }
    }
    uint64_t key[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i)
        key[i] = e0 + i < a.n_exp && (keep >> i & 1) ? route_key(c[i]) : 0;

    // lane t's result: slot my_slot of lane my_lane
    int my_lane = 0, my_slot = 0;
    bool near = false;
    {
        uint32_t k[NI], last = 0;
#pragma unroll
        for (int i = 0; i < NI; ++i)
            k[i] = key[i] ? ((uint32_t)(key[i] >> 32) & ~(uint32_t)(NI - 1)) | (NI - 1 - i) : 0u;
        for (int t = 0; t <= a.topk; ++t) {       // one more than needed: the best that is left
            uint32_t best = k[0];
#pragma unroll
            for (int i = 1; i < NI; ++i)
                best = best > k[i] ? best : k[i];
            const uint32_t top = wave_max(best);
            near |= t > 0 && top != 0 && (top ^ last) < (uint32_t)NI;
            last = top;
            const int w = __ffsll((unsigned long long)__ballot(best == top)) - 1;
#pragma unroll
            for (int i = 0; i < NI; ++i)
                k[i] = lane == w && k[i] == top ? 0u : k[i];
            if (lane == t) {
                my_lane = w;
                my_slot = NI - 1 - (int)(top & (NI - 1));
            }
        }
    }
    if (near) {
        for (int t = 0; t < a.topk; ++t) {
            uint64_t k = key[0];
            int at = 0;
#pragma unroll
            for (int i = 1; i < NI; ++i)
                if (key[i] > k) {
                    k = key[i];
                    at = i;
                }
            const int w = best_lane(k);
            const int wi = __builtin_amdgcn_readlane(at, w);
#pragma unroll
            for (int i = 0; i < NI; ++i)
                key[i] = lane == w && i == wi ? 0 : key[i];
            if (lane == t) {
                my_lane = w;
                my_slot = wi;
            }
        }
    }
    double mine = 0.0;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const double v = __shfl(s[i], my_lane);
        mine = i == my_slot ? v : mine;
    }
    mine = lane < a.topk ? mine : 0.0;
    if (a.renorm) {
        const double total = wave_sum(mine);
        mine = total == 0.0 ? 0.0 : mine / total;
    }
    if (lane < a.topk) {
        a.ids[r * a.topk + lane] = NI * my_lane + my_slot;
        a.wts[r * a.topk + lane] = (float)(mine * (double)a.scale);
    }
}

int launch_route(const RouteArgs &args, void *stream)
{
    RouteArgs a = args;
    const int lanes = (a.n_exp + 63) / 64;
    const int ni = lanes <= 1 ? 1 : lanes <= 2 ? 2 : lanes <= 4 ? 4 : lanes <= 8 ? 8 : 16;
    const int size = a.n_exp / a.n_group, run = size / ni;
    a.run_log2 = -1;                              // log2 of the lanes of a group, if it is a run of 2^k
    if (size % ni == 0 && (run & (run - 1)) == 0)
        for (a.run_log2 = 0; 1 << a.run_log2 < run;)
            ++a.run_log2;
    void (*k)(RouteArgs) = ni == 1 ? k_route<1> : ni == 2 ? k_route<2> : ni == 4 ? k_route<4> : ni == 8 ? k_route<8>
                                                                                                : k_route<16>;
    hipLaunchKernelGGL(k, dim3((unsigned)((a.n_rows + 3) / 4)), dim3(256), 0, static_cast<hipStream_t>(stream), a);
    return (int)hipGetLastError();
}

}  // namespace qg
