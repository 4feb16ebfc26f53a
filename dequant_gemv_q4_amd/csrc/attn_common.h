// attn_common.h -- device helpers of the paged cache and the attention kernels.
#pragma once

#include <hip/hip_runtime.h>

#include "attn_internal.h"

namespace qg {

typedef _Float16 ah8 __attribute__((ext_vector_type(8)));
typedef __bf16 ab8 __attribute__((ext_vector_type(8)));
typedef float af4 __attribute__((ext_vector_type(4)));
typedef float af16 __attribute__((ext_vector_type(16)));
typedef uint32_t au4 __attribute__((ext_vector_type(4)));

// Pieces an f32 value (a scaled query, a probability) is split into for the products with f16 / bf16
// operands: two f16 hold 22 of its 24 bits, three bf16 all of them.  (Two bf16, 2^-18, left
// attention outputs 2.4e-6 off in the root mean square where f32 sums leave 0.7e-6.)
template <int T> constexpr int PIECES = T == KV_F16 ? 2 : 3;

// Two floats rounded to nearest-even to the cache's type, packed (a in the low half): one
// instruction for either type.
template <int T>
__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    typedef float f2 __attribute__((ext_vector_type(2)));
    typedef _Float16 h2 __attribute__((ext_vector_type(2)));
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    const f2 v = {a, b};
    if constexpr (T == KV_F16)
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, h2));
    else
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, b2));
}
template <int T>
__device__ __forceinline__ float low_of(uint32_t p)
{
    if constexpr (T == KV_F16)
        return (float)__builtin_bit_cast(_Float16, (uint16_t)(p & 0xFFFFu));
    else
        return __builtin_bit_cast(float, p << 16);
}
template <int T>
__device__ __forceinline__ float high_of(uint32_t p)
{
    if constexpr (T == KV_F16)
        return (float)__builtin_bit_cast(_Float16, (uint16_t)(p >> 16));
    else
        return __builtin_bit_cast(float, p & 0xFFFF0000u);
}

// Eight floats as operands whose sum is the value.
template <int T>
__device__ __forceinline__ void split8(const float (&v)[8], au4 (&out)[PIECES<T>])
{
    float r[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
        r[e] = v[e];
#pragma unroll
    for (int i = 0; i < PIECES<T>; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t p = pack2<T>(r[2 * e], r[2 * e + 1]);
            out[i][e] = p;
            if (i + 1 < PIECES<T>) {
                r[2 * e] = fmaf(low_of<T>(p), -1.0f, r[2 * e]);     // f16: one instruction
                r[2 * e + 1] = fmaf(high_of<T>(p), -1.0f, r[2 * e + 1]);
            }
        }
}

// D += A B on the matrix cores, operands as raw dwords.
template <int T>
__device__ __forceinline__ af4 mm16(au4 a, au4 b, af4 c)
{
    if constexpr (T == KV_F16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(ah8, a),
                                                      __builtin_bit_cast(ah8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(ab8, a),
                                                       __builtin_bit_cast(ab8, b), c, 0, 0, 0);
}
template <int T>
__device__ __forceinline__ af16 mm32(au4 a, au4 b, af16 c)
{
    if constexpr (T == KV_F16)
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(ah8, a),
                                                      __builtin_bit_cast(ah8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(ab8, a),
                                                       __builtin_bit_cast(ab8, b), c, 0, 0, 0);
}

// Combine across lanes l, l ^ 32 (or l ^ 16): every lane gets the result.
__device__ __forceinline__ float max_x32(float v)
{
    const uint32_t b = __builtin_bit_cast(uint32_t, v);
    const auto s = __builtin_amdgcn_permlane32_swap(b, b, false, false);
    const uint32_t s0 = s[0], s1 = s[1];
    return fmaxf(__builtin_bit_cast(float, s0), __builtin_bit_cast(float, s1));
}
__device__ __forceinline__ float max_x16(float v)
{
    const uint32_t b = __builtin_bit_cast(uint32_t, v);
    const auto s = __builtin_amdgcn_permlane16_swap(b, b, false, false);
    const uint32_t s0 = s[0], s1 = s[1];
    return fmaxf(__builtin_bit_cast(float, s0), __builtin_bit_cast(float, s1));
}
__device__ __forceinline__ float sum_x32(float v)
{
    const uint32_t b = __builtin_bit_cast(uint32_t, v);
    const auto s = __builtin_amdgcn_permlane32_swap(b, b, false, false);
    const uint32_t s0 = s[0], s1 = s[1];
    return __builtin_bit_cast(float, s0) + __builtin_bit_cast(float, s1);
}
__device__ __forceinline__ float sum_x16(float v)
{
    const uint32_t b = __builtin_bit_cast(uint32_t, v);
    const auto s = __builtin_amdgcn_permlane16_swap(b, b, false, false);
    const uint32_t s0 = s[0], s1 = s[1];
    return __builtin_bit_cast(float, s0) + __builtin_bit_cast(float, s1);
}

// Power of two that brings a query row's largest |value| to [2^13, 2^14): both f16 pieces of every
// value then keep their bits (the second one down to 2^-38 of the row's largest).  bf16 has the
// range of f32 and is not scaled.  A row of zeros, infinities or NaN keeps the factor 1.
template <int T>
__device__ __forceinline__ float q_scale(float amax)
{
    if constexpr (T != KV_F16)
        return 1.0f;
    if (!(amax > 0.f) || !(amax < INFINITY))
        return 1.0f;
    int e = 0;
    frexpf(amax, &e);
    const int k = 14 - e;
    return ldexpf(1.0f, k < 126 ? k : 126);
}

// Bits 15 and 31 set where a half of the pair is an infinity or NaN.
template <int T>
__device__ __forceinline__ uint32_t nonfinite2(uint32_t v)
{
    return T == KV_F16 ? ((v & 0x7C007C00u) + 0x04000400u) & 0x80008000u
                       : ((v & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
}

constexpr float LOG2E = 1.44269504088896340736f;

}  // namespace qg
