// route_kernels.hip -- routing of rows to experts: scores, groups, top-k, weights.
//
// s = softmax(z) or sigmoid(z) over a row's experts, choice c = s + bias; the topk_group groups
// with the largest sum of their best group_top c stay; the topk largest c among them, ties to the
// lower index; weights s (renormalised) * scale.
//
// One wave per row, expert e = lane + 64 i in register i.  Scores and choices are f64: two choices
// that differ by less than an f32 rounding (a bias near the scores' own spacing) must come out in
// their true order, and gfx950 runs f64 at the f32 rate.  A choice is compared as the unsigned
// image of its bits (order-preserving), 0 meaning "not selectable".
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

// The wave's largest key and the lowest index holding it.
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

template <int NI>
__global__ __launch_bounds__(256) void k_route(RouteArgs a)
{
    __shared__ double sc[4][64 * NI];
    __shared__ uint8_t keep[4][64 * NI];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int64_t r = (int64_t)blockIdx.x * 4 + wave;
    if (r >= a.n_rows)
        return;                                   // no workgroup barrier below
    const float *zr = a.z + r * a.n_exp;
    float z[NI];
    double s[NI];
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int e = lane + 64 * i;
        z[i] = e < a.n_exp ? zr[e] : -INFINITY;
        m = fmaxf(m, z[i]);
    }
    if (a.sigmoid) {
#pragma unroll
        for (int i = 0; i < NI; ++i)
            s[i] = 1.0 / (1.0 + exp(-(double)z[i]));
    } else {
#pragma unroll
        for (int x = 32; x; x >>= 1)
            m = fmaxf(m, __shfl_xor(m, x));
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            s[i] = lane + 64 * i < a.n_exp ? exp((double)z[i] - (double)m) : 0.0;
            sum += s[i];
        }
#pragma unroll
        for (int x = 32; x; x >>= 1)
            sum += __shfl_xor(sum, x);
#pragma unroll
        for (int i = 0; i < NI; ++i)
            s[i] /= sum;
    }
    uint64_t key[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int e = lane + 64 * i;
        const double c = a.bias && e < a.n_exp ? s[i] + (double)a.bias[e] : s[i];
        key[i] = e < a.n_exp ? route_key(c) : 0;
        sc[wave][e] = c;
    }
    auto wave_sync = []() {
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    };
    if (a.n_group > 1) {
        wave_sync();
        const int size = a.n_exp / a.n_group;
        uint64_t gk[NI];
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int g = lane + 64 * i;
            gk[i] = 0;
            keep[wave][g] = 0;
            if (g < a.n_group) {
                double b1 = -INFINITY, b2 = -INFINITY;
                for (int j = 0; j < size; ++j) {
                    double c = sc[wave][g * size + j];
                    c = c == c ? c : -INFINITY;
                    b2 = fmax(b2, fmin(b1, c));
                    b1 = fmax(b1, c);
                }
                gk[i] = route_key(a.group_top == 2 ? b1 + b2 : b1);
            }
        }
        for (int t = 0; t < a.topk_group; ++t) {
            uint64_t k = 0;
            int idx = 0x7fffffff;
#pragma unroll
            for (int i = 0; i < NI; ++i)
                if (gk[i] > k) {
                    k = gk[i];
                    idx = lane + 64 * i;
                }
            wave_best(k, idx);
#pragma unroll
            for (int i = 0; i < NI; ++i)
                if (idx == lane + 64 * i) {
                    gk[i] = 0;
                    keep[wave][idx] = 1;
                }
        }
        wave_sync();
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int e = lane + 64 * i;
            if (e < a.n_exp && !keep[wave][e / size])
                key[i] = 0;
        }
    }
    double total = 0.0, mine = 0.0;
    int my_id = 0;
    for (int t = 0; t < a.topk; ++t) {
        uint64_t k = 0;
        int idx = 0x7fffffff;
        double sv = 0.0;
#pragma unroll
        for (int i = 0; i < NI; ++i)
            if (key[i] > k) {
                k = key[i];
                idx = lane + 64 * i;
            }
        wave_best(k, idx);
#pragma unroll
        for (int i = 0; i < NI; ++i)
            if (idx == lane + 64 * i) {
                key[i] = 0;
                sv = s[i];
            }
        sv = __shfl(sv, idx & 63);
        total += sv;
        if (lane == t) {
            mine = sv;
            my_id = idx;
        }
    }
    if (lane < a.topk) {
        if (a.renorm)
            mine = total == 0.0 ? 0.0 : mine / total;
        a.ids[r * a.topk + lane] = my_id;
        a.wts[r * a.topk + lane] = (float)(mine * (double)a.scale);
    }
}

int launch_route(const RouteArgs &a, void *stream)
{
    hipStream_t s = static_cast<hipStream_t>(stream);
    const dim3 grid((unsigned)((a.n_rows + 3) / 4));
    const int ni = (a.n_exp + 63) / 64;
    auto k = ni <= 1 ? k_route<1> : ni <= 2 ? k_route<2> : ni <= 4 ? k_route<4> : ni <= 8 ? k_route<8>
                                                                                      : k_route<16>;
    hipLaunchKernelGGL(k, grid, dim3(256), 0, s, a);
    return (int)hipGetLastError();
}

}  // namespace qg
