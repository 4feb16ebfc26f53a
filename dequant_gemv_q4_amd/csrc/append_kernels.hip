// append_kernels.hip -- from the fused QKV output to the cache: norm and rotation of the Q and K heads,
// and new rows of K and V in pages of any type; and new rows alone in 8-bit pages.
//
// A workgroup takes one head of one block of 16 or 32 positions (at most a page) of a sequence: a KV head
// (its K, then its V) or a Q head.  A row of a head is shared by LPR lanes, four channels each, so a wave
// holds 64 / LPR rows and reads them in runs of whole heads; the sums and maxima of a row go over those
// lanes.  The channel that a channel is rotated with is read again instead of exchanged (the line is in the
// L1).
//
// K is turned in 64 bits and rounded once: it ends in 3 to 10 bits, and which of two neighbours a value
// near their middle takes must not depend on the order of the sums (gfx950 runs f64 at the f32 rate).  Codes
// are those of the exact quotient x / d: the quotient by multiplication is off by one step at most, and its
// remainder x - n d is exact (f32: n has 7 bits, and the remainder is a multiple of half d's last bit not
// above d), so it decides, ties included.  V goes through LDS to lie transposed in the page, 16 bytes of a
// channel at a time; a piece with positions that are not new is written element by element.
#include <hip/hip_runtime.h>

#include <float.h>

#include "attn_common.h"

namespace qg {

// f64 to f32 so that a further rounding to at most 22 bits gives that of the f64 value: truncated towards
// the odd neighbour.
__device__ __forceinline__ float to_odd(double x)
{
    const float f = (float)x;
    const double r = x - (double)f;
    if (r == 0.0 || !(fabs(r) <= DBL_MAX))
        return f;
    const uint32_t b = __builtin_bit_cast(uint32_t, f);
    if (b & 1u)
        return f;
    return __builtin_bit_cast(float, (r < 0.0) == (x < 0.0) ? b + 1u : b - 1u);
}
__device__ __forceinline__ float to_odd(float x) { return x; }

__device__ __forceinline__ float fma_of(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ double fma_of(double a, double b, double c) { return fma(a, b, c); }

// Combine over the LPR lanes of a row; every lane gets the result.
template <int LPR, class R, class F>
__device__ __forceinline__ R over_row(R v, F f)
{
#pragma unroll
    for (int m = 1; m < LPR; m *= 2)
        v = f(v, __shfl_xor(v, m, 64));
    return v;
}

// The scale of a row from its largest |value| (not finite: NaN).
template <int T, class R>
__device__ __forceinline__ float scale_of(R amax)
{
    if (!(amax <= (R)FLT_MAX))
        return __builtin_nanf("");
    if constexpr (T == KV_I8) {
        return fmaxf((float)(amax / (R)127), 0x1p-126f);
    } else {
        // amax = m 2^e, m in [1/2, 1), and 448 = 7/8 2^9
        int e = 0;
        const R m = sizeof(R) == 8 ? (R)frexp((double)amax, &e) : (R)frexpf((float)amax, &e);
        const int k = e - 9 + (m > (R)0.875 ? 1 : 0);
        return ldexpf(1.0f, amax == (R)0 || k < -126 ? -126 : k);
    }
}

// The codes of four values of a row with scale d, a byte each.
template <int T, class R>
__device__ __forceinline__ uint32_t codes_of(const R (&x)[4], float d)
{
    if (d != d)
        return 0u;
    const R dd = (R)d, inv = (R)1 / dd;
    if constexpr (T == KV_I8) {
        uint32_t out = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const R n = __builtin_elementwise_rint(x[e] * inv), r = fma_of(-n, dd, x[e]), two = r + r;
            int i = (int)n;
            if (two > dd || (two == dd && (i & 1)))
                ++i;
            if (-two > dd || (-two == dd && (i & 1)))
                --i;
            out |= (uint32_t)(i & 0xFF) << (8 * e);
        }
        return out;
    } else {
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            y[e] = to_odd(x[e] * inv);                   // d is a power of two
        int p = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
        p = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], p, true);
        return (uint32_t)p;
    }
}

// Channels of a head, rounded up to a power of two lanes of four.
constexpr int lanes_per_row(int hd) { return hd <= 64 ? 16 : hd <= 128 ? 32 : 64; }

// TURN: norms and rotation (and Q heads); else K and V as they come.  VEC: rope_half is a multiple of four.
template <int T, int BL, int LPR, bool TURN, bool VEC>
__global__ __launch_bounds__(256) void k_qkv_append(QkvArgs a)
{
    typedef typename std::conditional<TURN, double, float>::type RK;
    constexpr int BLOCK = 1 << BL, ROWS = 256 / LPR, SIZE = kv_bytes(T) ? 1 : 2;
    constexpr int STRIDE = BLOCK * SIZE + 4;               // bytes of a channel in LDS
    __shared__ __attribute__((aligned(16))) uint8_t s_v[4 * LPR * STRIDE];
    const KvArgs &c = a.c;
    const int tid = threadIdx.x, role = blockIdx.y, j = tid % LPR, row = tid / LPR, ch = 4 * j;
    const bool in = ch < c.hd;
    AppendBlock w;
    if (!append_block<BL>(c, w))
        return;
    int from = w.from, to = w.to;
    if (TURN && a.half > 0 && w.t0 + to > a.rope_rows) {
        if (tid == 0)
            atomicOr(c.err, 1u);
        to = (int)max(a.rope_rows - w.t0, (int64_t)0);
    }
    if (from >= to)
        return;

    auto load4 = [&](const float *p, float (&x)[4]) {
        const float4 v = *reinterpret_cast<const float4 *>(p);
        x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    };
    // four channels of a head at position t0 + t, normalised and rotated
    auto turned = [&](const float *x, const float *gamma, int t, auto one) {
        typedef decltype(one) R;
        struct Four {
            R v[4];
        } r;
        float y[4] = {0.f, 0.f, 0.f, 0.f}, z[4] = {0.f, 0.f, 0.f, 0.f}, gy[4], gz[4];
        // channel ch + e is turned with the one `other` away
        const int h = a.half;
        float cs[4], sn[4];
        int other[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int k = ch + e, at = VEC ? ch : k;
            other[e] = in && at < 2 * h ? (at < h ? h : -h) : 0;
            gy[e] = gz[e] = 1.f;
            cs[e] = 1.f;
            sn[e] = 0.f;
        }
        if (in) {
            load4(x + ch, y);
            if (gamma)
                load4(gamma + ch, gy);
            const int64_t turn = (w.t0 + t) * h;
            if constexpr (VEC) {
                if (other[0]) {
                    load4(x + ch + other[0], z);
                    if (gamma)
                        load4(gamma + ch + other[0], gz);
                    const int k = other[0] > 0 ? ch : ch - h;
                    load4(a.cos + turn + k, cs);
                    load4(a.sin + turn + k, sn);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (other[e]) {
                        z[e] = x[ch + e + other[e]];
                        if (gamma)
                            gz[e] = gamma[ch + e + other[e]];
                        const int k = other[e] > 0 ? ch + e : ch + e - h;
                        cs[e] = a.cos[turn + k];
                        sn[e] = a.sin[turn + k];
                    }
            }
        }
        R scale = (R)1;
        if (gamma) {
            R ss = (R)0;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                ss = fma_of((R)y[e], (R)y[e], ss);
            ss = over_row<LPR>(ss, [](R u, R v) { return u + v; });
            const R mean = ss / (R)c.hd + (R)a.eps;
            scale = (R)1 / (sizeof(R) == 8 ? (R)sqrt((double)mean) : (R)sqrtf((float)mean));
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const R u = gamma ? (R)y[e] * (R)gy[e] * scale : (R)y[e], v = gamma ? (R)z[e] * (R)gz[e] * scale : (R)z[e];
            r.v[e] = other[e] ? fma_of(u, (R)cs[e], other[e] > 0 ? -v * (R)sn[e] : v * (R)sn[e]) : u;
        }
        return r;
    };

    if (role >= c.nkv) {                                   // a Q head
        const int h = role - c.nkv;
        for (int t = from + row; t < to; t += ROWS) {
            const auto r = turned(a.q + (w.row0 + t) * a.stride + (int64_t)h * c.hd, a.q_gamma, t, 1.0f);
            if (in)
                *reinterpret_cast<float4 *>(a.qo + (w.row0 + t) * a.qo_stride + (int64_t)h * c.hd + ch) =
                    make_float4(r.v[0], r.v[1], r.v[2], r.v[3]);
        }
        return;
    }

    const int page = append_page(c, w), h = role;
    if (page < 0) {
        if (tid == 0 && h == 0)
            atomicOr(c.err, 1u);
        return;
    }
    const int slot = (int)(w.t0 & ((1 << c.ps_log2) - 1));
    const int64_t base = (int64_t)page * c.page_stride + (int64_t)h * c.block;
    const int64_t codes = (int64_t)c.hd << c.ps_log2;      // elements before an 8-bit block's scales

    // K: a row's codes lie side by side
    for (int t = from + row; t < to; t += ROWS) {
        const float *src = a.k + (w.row0 + t) * a.stride + (int64_t)h * c.hd;
        RK x[4] = {0, 0, 0, 0};
        if constexpr (TURN) {
            const auto r = turned(src, a.k_gamma, t, 1.0);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                x[e] = r.v[e];
        } else if (in) {
            float y[4];
            load4(src + ch, y);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                x[e] = y[e];
        }
        const int64_t at = base + (int64_t)(slot + t) * c.hd + ch;
        if constexpr (SIZE == 1) {
            RK top = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const RK v = x[e] < 0 ? -x[e] : x[e];
                top = v <= top ? top : v <= (RK)FLT_MAX ? v : (RK)INFINITY;
            }
            top = over_row<LPR>(top, [](RK u, RK v) { return u > v ? u : v; });
            const float d = scale_of<T>(top);
            if (in)
                *reinterpret_cast<uint32_t *>(c.k8() + at) = codes_of<T>(x, d);
            if (j == 0)
                *reinterpret_cast<float *>(c.k8() + base + codes + 4 * (slot + t)) = d;
        } else if (in) {
            uint2 v;
            v.x = pack2<T>(to_odd(x[0]), to_odd(x[1]));
            v.y = pack2<T>(to_odd(x[2]), to_odd(x[3]));
            *reinterpret_cast<uint2 *>(c.k + at) = v;
        }
    }

    // V: by rows into LDS, by channels out of it
    for (int t = from + row; t < to; t += ROWS) {
        float x[4] = {0.f, 0.f, 0.f, 0.f};
        if (in)
            load4(a.v + (w.row0 + t) * a.stride + (int64_t)h * c.hd + ch, x);
        if constexpr (SIZE == 1) {
            float top = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                top = fabsf(x[e]) <= top ? top : fabsf(x[e]) <= FLT_MAX ? fabsf(x[e]) : INFINITY;
            top = over_row<LPR>(top, [](float u, float v) { return u > v ? u : v; });
            const float d = scale_of<T>(top);
            const uint32_t v = codes_of<T>(x, d);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                s_v[(ch + e) * STRIDE + t] = (uint8_t)(v >> (8 * e));
            if (j == 0)
                *reinterpret_cast<float *>(c.v8() + base + codes + 4 * (slot + t)) = d;
        } else {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t v = pack2<T>(x[2 * e], x[2 * e + 1]);
                *reinterpret_cast<uint16_t *>(s_v + (ch + 2 * e) * STRIDE + 2 * t) = (uint16_t)v;
                *reinterpret_cast<uint16_t *>(s_v + (ch + 2 * e + 1) * STRIDE + 2 * t) = (uint16_t)(v >> 16);
            }
        }
    }
    __syncthreads();
    constexpr int PER = 16 / SIZE, PIECES_V = BLOCK / PER;  // positions of a piece, pieces of a channel
    for (int x = tid; x < c.hd * PIECES_V; x += 256) {
        const int d = x / PIECES_V, t = PER * (x % PIECES_V);
        if (t >= to || t + PER <= from)
            continue;
        const uint8_t *src = s_v + d * STRIDE + t * SIZE;
        uint8_t *dst = c.v8() + (base + ((int64_t)d << c.ps_log2) + slot + t) * SIZE;
        if (t >= from && t + PER <= to) {
            const uint32_t *p = reinterpret_cast<const uint32_t *>(src);
            *reinterpret_cast<au4 *>(dst) = au4{p[0], p[1], p[2], p[3]};
        } else {
            for (int e = max(from - t, 0); e < min(to - t, PER); ++e)
                if constexpr (SIZE == 1)
                    dst[e] = src[e];
                else
                    reinterpret_cast<uint16_t *>(dst)[e] = reinterpret_cast<const uint16_t *>(src)[e];
        }
    }
}

template <int T, int BL, bool TURN>
static void launch_block(const QkvArgs &a, dim3 grid, hipStream_t s)
{
    const bool vec = a.half % 4 == 0;
    void (*k)(QkvArgs) = nullptr;
#define QG_APPEND_L(L) k = !TURN || vec ? k_qkv_append<T, BL, L, TURN, true> : k_qkv_append<T, BL, L, TURN, !TURN>
    switch (lanes_per_row(a.c.hd)) {
    case 16: QG_APPEND_L(16); break;
    case 32: QG_APPEND_L(32); break;
    default: QG_APPEND_L(64); break;
    }
#undef QG_APPEND_L
    hipLaunchKernelGGL(k, grid, dim3(256), 0, s, a);
}

int launch_qkv_append(int kv_type, bool turn, const QkvArgs &a, void *stream)
{
    const int bl = a.c.ps_log2 < 5 ? 4 : 5;
    const int64_t blocks = a.c.q_start ? (a.c.n_rows >> bl) + 2 * (int64_t)a.c.n_seq : a.c.n_seq;
    const dim3 grid((unsigned)blocks, (unsigned)(a.c.nkv + (turn ? a.nq : 0)));
    hipStream_t s = static_cast<hipStream_t>(stream);
#define QG_APPEND(T)                                                       \
    if (turn)                                                              \
        bl == 4 ? launch_block<T, 4, true>(a, grid, s) : launch_block<T, 5, true>(a, grid, s); \
    else                                                                   \
        bl == 4 ? launch_block<T, 4, false>(a, grid, s) : launch_block<T, 5, false>(a, grid, s)
    switch (kv_type) {
    case KV_I8: QG_APPEND(KV_I8); break;
    case KV_F8: QG_APPEND(KV_F8); break;
    case KV_F16: bl == 4 ? launch_block<KV_F16, 4, true>(a, grid, s) : launch_block<KV_F16, 5, true>(a, grid, s); break;
    default: bl == 4 ? launch_block<KV_BF16, 4, true>(a, grid, s) : launch_block<KV_BF16, 5, true>(a, grid, s); break;
    }
#undef QG_APPEND
    return (int)hipGetLastError();
}

}  // namespace qg
