// attn_bytes.h -- device helpers of the attention over 8-bit pages.
//
// A cached value is d * code with d one f32 scale for a position of a head, so scores are
// (q . code) d^K scale and outputs sum p (d^V code): codes enter the products as f16 (an e4m3 and a signed
// byte are one exactly), the scales the f32 scores and weights.  Queries and weights are two f16 pieces, as
// over f16 pages.
//
// What has to fit f16 is the weight times the scale of V, w = p d^V.  The scales are taken relative to 2^r, r
// a whole number that follows the largest scale that any column of a wave has met, and a column keeps the exponent
// `top` of the largest relative scale that it has seen (at least LEAST_TOP): its shift puts the largest p at
// 2^(LIFT - top), so that w is at most 2^LIFT when the shift moves and under 2^TOP afterwards.  When r moves up,
// a column's top goes down and its shift up by as much (rescaled), so that what it weighs from then on is as
// large as before; left alone, with V 2^29 and then 2^31 times larger than at first, the last weights kept four
// bits.  Of w 2^-25 is lost at most: 2^-35 of the largest weight times the largest scale that the column sees, as
// long as that scale is at least 2^LEAST_TOP of the largest that another column of the wave has seen.  Sums of p
// stay in f32: p is at most 2^(TOP - LEAST_TOP) = 2^96, of 2^24 positions 2^120.
#pragma once

#include <utility>

#include "attn_common.h"

namespace qg {

constexpr float LIFT8 = LIFT<KV_F16>, TOP8 = TOP<KV_F16>;
constexpr float LEAST_TOP = -80.0f;            // so far below 2^r, scales lose bits instead
constexpr float R_SLACK = 30.0f;               // 2^r moves when a scale is so far above it
constexpr float MOST_SUM = 114.0f;             // the exponent up to which a move of 2^r may raise a sum of weights
// Raw products are below 2^32 (queries to 2^14 log2 e, codes to 448, 256 channels): times K_ROOM of any scale of K
// they stay within f32.
constexpr float K_ROOM = 0x1p-32f;

// Sixteen codes as f16, in order.
template <int T>
__device__ __forceinline__ void halves_of(au4 x, au4 &lo, au4 &hi)
{
    typedef _Float16 h2 __attribute__((ext_vector_type(2)));
    uint32_t out[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (T == KV_F8) {
            out[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(x[i], 1.0f, false));
            out[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(x[i], 1.0f, true));
        } else {
            // 1024 + (128 + code) as an f16 is the byte below 0x64
            const uint32_t y = x[i] ^ 0x80808080u;
            const h2 off = {(_Float16)1152.0f, (_Float16)1152.0f};
            const h2 a = __builtin_bit_cast(h2, __builtin_amdgcn_perm(0x64646464u, y, 0x04010400u)) - off;
            const h2 b = __builtin_bit_cast(h2, __builtin_amdgcn_perm(0x64646464u, y, 0x04030402u)) - off;
            out[2 * i] = __builtin_bit_cast(uint32_t, a);
            out[2 * i + 1] = __builtin_bit_cast(uint32_t, b);
        }
    }
    lo = au4{out[0], out[1], out[2], out[3]};
    hi = au4{out[4], out[5], out[6], out[7]};
}

// The value of lane E of each 16 lanes.
template <int E>
__device__ __forceinline__ float lane_of_16(float v)
{
    return __builtin_bit_cast(float,
                              __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x150 + E, 0xF, 0xF, true));
}
// An element of a register vector.
template <class V>
struct Ref {
    V &v;
    int e;
    __device__ __forceinline__ Ref &operator*=(float f)
    {
        v[e] *= f;
        return *this;
    }
};
// x(e) *= lane e's v, of 16.
template <int... E, class X>
__device__ __forceinline__ void times_lanes(X &&x, float v, std::integer_sequence<int, E...>)
{
    ((x(E) *= lane_of_16<E>(v)), ...);
}
template <class X>
__device__ __forceinline__ void times_lanes(X &&x, float v)
{
    times_lanes(x, v, std::make_integer_sequence<int, 16>());
}
template <int... E, class X>
__device__ __forceinline__ void each_lane(X &&x, float v, std::integer_sequence<int, E...>)
{
    ((x(E, lane_of_16<E>(v))), ...);
}
// x(e, lane e's v) for e < 16.
template <class X>
__device__ __forceinline__ void each_lane(X &&x, float v)
{
    each_lane(x, v, std::make_integer_sequence<int, 16>());
}

// The exponent e of the least power of two above v (0: very low).
__device__ __forceinline__ float exponent_above(float v)
{
    return v > 0.f ? (float)__builtin_amdgcn_frexp_expf(v) : -200.0f;
}

// shift_of for weights that end at 2^(TOP8 - top).  Where scores are so large that LIFT8 - top - score is
// rounded too far up, one rounding step less than -top - score is as good.
__device__ __forceinline__ float shift8_of(float top_score, float top)
{
    const float r = LIFT8 - top - top_score;
    return r + top_score > TOP8 - top ? -top_score - top - fabsf(top_score) * 0x1p-23f : r;
}

// A column when its wave rescales: because a score would bring a weight above 2^TOP, or because the reference moves
// from 2^r up to 2^to (else to = r).  top includes the scales of this step; score is the largest of its
// scores, sum the exponent of its sum of weights, over its lanes.  As the reference moves, the shift rises by what
// top falls, but not so far that the sum could reach f32's end: a column whose sum would has weighed positions with
// small scales by 2^92 or more (2^114 over the 2^22 positions of a wave), and needs no further bits for what comes.
// Where scores are so large that the shift would be rounded by more than a quarter, it stays.  (One branch for both
// reasons: with one each, heads of 256 spilled, 4000 rows, 16 / 8 heads, I8, 436 us against 368.)
struct Rescaled {
    float top, shift, l, o;                    // top and shift from now on; factors of the sum and of O
};
__device__ __forceinline__ Rescaled rescaled(float r, float to, float top, float shift, float score, float sum)
{
    Rescaled x;
    x.top = r == to ? top : fmaxf(top + (r - to), LEAST_TOP);
    const float rise = fmaxf(fminf(fminf(top, R_SLACK) - x.top, MOST_SUM - sum), 0.f);
    x.shift = fminf(fabsf(shift) < 0x1p22f ? shift + rise : shift, shift8_of(score, x.top));
    const float by = x.shift - shift;
    x.l = __builtin_amdgcn_exp2f(by);
    x.o = __builtin_amdgcn_exp2f(by + (r - to));
    return x;
}

// A part of a column's positions is held as its mean (weighted by the weights), the exponent m of its weights
// and their sum l; parts k join by the factors l_k 2^(m_k - max m) over their sum.  What a part counts for is
// in l alone, so that a mean near the end of f32 never overflows; 0 x NaN keeps a NaN that was seen.
struct Factors {
    float m, l;
};
template <int N>
__device__ __forceinline__ Factors join_factors(const float (&m)[N], const float (&l)[N], int n, float (&f)[N])
{
    Factors r = {-INFINITY, 0.f};
#pragma unroll
    for (int k = 0; k < N; ++k)
        if (k < n)
            r.m = fmaxf(r.m, m[k]);
#pragma unroll
    for (int k = 0; k < N; ++k)
        if (k < n) {
            f[k] = l[k] * join_weight(m[k], r.m);
            r.l += f[k];
        }
    const float inv = inverse_sum(r.l);
#pragma unroll
    for (int k = 0; k < N; ++k)
        if (k < n)
            f[k] *= inv;
    return r;
}

}  // namespace qg
