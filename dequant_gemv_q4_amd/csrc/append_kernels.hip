// append_kernels.hip -- from the fused QKV output to the cache: norm and rotation of the Q and K heads,
// and new rows of K and V in pages of any type; and new rows alone in 8-bit pages.
//
// A workgroup takes K or V of a KV head, or four Q heads, of one block of 16 or 32 positions (at most a page)
// of a sequence.  A row of a head is shared by LPR lanes, four channels each, so a wave holds 64 / LPR rows
// and reads them in runs of whole heads; the sums and maxima of a row go over those lanes.  The channel that a
// channel is rotated with is read again instead of exchanged (the line is in the L1; a swap of half rows took
// as long).
//
// K is turned in 64 bits and rounded once: it ends in 3 to 10 bits, and which of two neighbours a value
// near their middle takes must not depend on the order of the sums (gfx950 runs f64 at the f32 rate).  Codes
// are those of the exact quotient x / d: taken in f32, and again by the remainder where that is too near to the
// middle of two.  V goes through LDS to lie transposed in the page, 16 bytes of a channel at a time; a piece with
// positions that are not new is written element by element.
//
// Bound by HBM: 8000 rows of 32 / 8 heads of 128 (349 MB read and written) take 72.4 us into I8 pages, 4.8 TB/s,
// 8000 rows of 8 heads of 128 alone into F8 (82 MB) 17.7 us, 4.7 TB/s, where a copy reaches 4.9.  One token 3.9 to
// 4.4 us, a launch.  Q in f64 as well, and one head a workgroup: 115 us for the first.
#include <hip/hip_runtime.h>

#include <float.h>

#include <type_traits>

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

// 1 / sqrt(x) to the last place or two, by a step of Newton's method from the instruction's value; f64 by two
// steps from the instruction's 2^-14 or better (an infinity or a zero stays with its answer).
__device__ __forceinline__ float inverse_root(float x)
{
    if (!(x > 0x1p-100f) || !(x <= FLT_MAX))
        return 1.0f / sqrtf(x);
    const float r = __builtin_amdgcn_rsqf(x);
    return fmaf(r * 0.5f, fmaf(-x * r, r, 1.0f), r);
}
__device__ __forceinline__ double inverse_root(double x)
{
    double r = __builtin_amdgcn_rsq(x);
    if (!(x > 0.0) || !(x <= DBL_MAX))
        return r;
#pragma unroll
    for (int i = 0; i < 2; ++i)
        r = fma(r * 0.5, fma(-x * r, r, 1.0), r);
    return r;
}

// A value of the lane that a DPP control names within 16 lanes.
template <int CTRL, class R>
__device__ __forceinline__ R moved(R v)
{
    if constexpr (sizeof(R) == 4) {
        return __builtin_bit_cast(R, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
    } else {
        const uint64_t b = __builtin_bit_cast(uint64_t, v);
        const uint32_t lo = moved<CTRL>((uint32_t)b), hi = moved<CTRL>((uint32_t)(b >> 32));
        return __builtin_bit_cast(R, (uint64_t)hi << 32 | lo);
    }
}
// v of lanes l and l ^ 16 (HALF: l ^ 32), combined.
template <bool HALF, class R, class F>
__device__ __forceinline__ R crossed(R v, F f)
{
    auto swap = [](uint32_t b) {
        if constexpr (HALF)
            return __builtin_amdgcn_permlane32_swap(b, b, false, false);
        else
            return __builtin_amdgcn_permlane16_swap(b, b, false, false);
    };
    if constexpr (sizeof(R) == 4) {
        const auto s = swap(__builtin_bit_cast(uint32_t, v));
        const uint32_t s0 = s[0], s1 = s[1];
        return f(__builtin_bit_cast(R, s0), __builtin_bit_cast(R, s1));
    } else {
        const uint64_t b = __builtin_bit_cast(uint64_t, v);
        const auto lo = swap((uint32_t)b), hi = swap((uint32_t)(b >> 32));
        const uint32_t l0 = lo[0], l1 = lo[1], h0 = hi[0], h1 = hi[1];
        return f(__builtin_bit_cast(R, (uint64_t)h0 << 32 | l0), __builtin_bit_cast(R, (uint64_t)h1 << 32 | l1));
    }
}
// Combine over the LPR lanes of a row; every lane gets the result (of sums, up to their order).
template <int LPR, class R, class F>
__device__ __forceinline__ R over_row(R v, F f)
{
    v = f(v, moved<0x121>(v));                             // row_ror 1, 2, 4, 8
    v = f(v, moved<0x122>(v));
    v = f(v, moved<0x124>(v));
    v = f(v, moved<0x128>(v));
    if constexpr (LPR >= 32)
        v = crossed<false>(v, f);
    if constexpr (LPR >= 64)
        v = crossed<true>(v, f);
    return v;
}

// The largest of the four |values| that a lane has of a row, over the row; not finite if one of them is not.
template <int LPR>
__device__ __forceinline__ float largest_of(const float (&x)[4])
{
    uint32_t top = 0;                                      // f32 in the order of their bits, NaN the largest
#pragma unroll
    for (int e = 0; e < 4; ++e)
        top = max(top, __builtin_bit_cast(uint32_t, x[e]) & 0x7FFFFFFFu);
    return __builtin_bit_cast(float, over_row<LPR>(top, [](uint32_t u, uint32_t v) { return u > v ? u : v; }));
}
template <int LPR>
__device__ __forceinline__ double largest_of(const double (&x)[4])
{
    double top = 0.0, sound = 0.0;                         // 0 times what is not finite is NaN
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        top = fmax(top, fabs(x[e]));
        sound = fma(x[e], 0.0, sound);
    }
    top = sound == sound ? top : (double)INFINITY;
    return over_row<LPR>(top, [](double u, double v) { return fmax(u, v); });
}

// The scale of a row from its largest |value| (not finite, or beyond f32: NaN).  The product with f64's 1 / 127
// rounds to the same f32 as the quotient of an f32: that is 2^-31 of itself from the middle of two f32 at least.
template <int T, class R>
__device__ __forceinline__ float scale_of(R amax)
{
    if (!(amax <= (R)FLT_MAX))
        return __builtin_nanf("");
    if constexpr (T == KV_I8) {
        return fmaxf((float)((double)amax * (1.0 / 127)), 0x1p-126f);
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
    const float inv = 1.0f / d;
    if constexpr (T == KV_I8) {
        int n[4];
        float off = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float u = (float)x[e] * inv, q = __builtin_rintf(u);
            n[e] = (int)q;
            off = fmaxf(off, fabsf(u - q));
        }
        // u is off by three roundings, 3 * 2^-24 * 127 < 2^-14: so near to the middle of two codes the remainder
        // of the nearer one decides, exact for an f32 (a multiple of half d's last bit not above d)
        if (__any(off > 0.5f - 0x1p-14f))
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const R r = fma_of(-(R)n[e], (R)d, x[e]), two = r + r;
                const bool odd = n[e] & 1;
                if (two > (R)d || (two == (R)d && odd))
                    ++n[e];
                else if (-two > (R)d || (-two == (R)d && odd))
                    --n[e];
            }
        return (uint32_t)(n[0] & 0xFF) | (uint32_t)(n[1] & 0xFF) << 8 | (uint32_t)(n[2] & 0xFF) << 16 |
               (uint32_t)n[3] << 24;
    } else {
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            y[e] = to_odd(x[e]) * inv;                   // d is a power of two
        int p = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
        p = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], p, true);
        return (uint32_t)p;
    }
}

// Channels of a head, rounded up to a power of two lanes of four.
constexpr int lanes_per_row(int hd) { return hd <= 64 ? 16 : hd <= 128 ? 32 : 64; }

constexpr int Q_HEADS = 4;                                 // of a workgroup, their loads in flight together

// TURN: norms and rotation (and Q heads); else K and V as they come.  VEC: rope_half is a multiple of four.
template <int T, int BL, int LPR, bool TURN, bool VEC>
__global__ __launch_bounds__(256) void k_qkv_append(QkvArgs a)
{
    typedef typename std::conditional<TURN, double, float>::type RK;
    constexpr int BLOCK = 1 << BL, ROWS = 256 / LPR, SIZE = kv_bytes(T) ? 1 : 2;
    constexpr int STRIDE = BLOCK * SIZE + 4;               // bytes of a channel in LDS
    __shared__ __attribute__((aligned(16))) uint8_t s_v[4 * LPR * STRIDE];
    const KvArgs &c = a.c;
    const int tid = threadIdx.x, j = tid % LPR, row = tid / LPR, ch = 4 * j;
    // roles of a block side by side: the workgroups at work read and write whole rows
    const int64_t all = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    const int id = (int)(all / a.roles), role = (int)(all - (int64_t)id * a.roles);
    const bool in = ch < c.hd;
    AppendBlock w;
    if ((!c.q_start && id >= c.n_seq) || !append_block<BL>(c, id, w))
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
    // channel ch + e is turned with the one other(e) away (0: not at all)
    auto other = [&](int e) {
        const int k = VEC ? ch : ch + e;
        return !TURN || !in || k >= 2 * a.half ? 0 : k < a.half ? a.half : -a.half;
    };
    // four channels, or those that they are turned with (left as they were where they are not)
    auto load = [&](const float *p, float (&x)[4]) {
        if (in)
            load4(p + ch, x);
    };
    auto load_other = [&](const float *p, float (&x)[4]) {
        if constexpr (VEC) {
            if (other(0))
                load4(p + ch + other(0), x);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (other(e))
                    x[e] = p[ch + e + other(e)];
        }
    };
    const double inv_hd = 1.0 / c.hd;
    // of four channels: the weights of the norm, and the factors of a channel and its other one at a position
    struct Weights {
        float y[4], z[4];
    };
    auto weights_of = [&](const float *gamma) {
        Weights g;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            g.y[e] = g.z[e] = 1.f;
        if (gamma) {
            load(gamma, g.y);
            load_other(gamma, g.z);
        }
        return g;
    };
    auto factors_of = [&](int t, const Weights &g, auto &fy, auto &fz) {
        typedef typename std::remove_reference<decltype(fy[0])>::type R;
        const int64_t at = (w.t0 + t) * a.half;
        float cs[4] = {1.f, 1.f, 1.f, 1.f}, sn[4] = {};
        if constexpr (VEC) {
            if (other(0)) {
                const int k = other(0) > 0 ? ch : ch - a.half;
                load4(a.cos + at + k, cs);
                load4(a.sin + at + k, sn);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (other(e)) {
                    const int k = ch + e + (other(e) > 0 ? 0 : other(e));
                    cs[e] = a.cos[at + k];
                    sn[e] = a.sin[at + k];
                }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            fy[e] = (R)g.y[e] * (R)cs[e];
            fz[e] = (R)g.z[e] * (R)(other(e) > 0 ? -sn[e] : sn[e]);
        }
    };
    // a head's four channels y (z: those they are turned with), normalised and turned
    auto turned = [&](const float (&y)[4], const float (&z)[4], bool norm, const auto &fy, const auto &fz, auto &out) {
        typedef typename std::remove_reference<decltype(out[0])>::type R;
        R scale = (R)1;
        if (norm) {
            R ss = (R)0;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                ss = fma_of((R)y[e], (R)y[e], ss);
            ss = over_row<LPR>(ss, [](R u, R v) { return u + v; });
            scale = inverse_root(fma_of(ss, (R)inv_hd, (R)a.eps));
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const R r = fma_of((R)y[e], fy[e], (R)z[e] * fz[e]);
            out[e] = norm ? r * scale : r;
        }
    };

    if (role >= 2 * c.nkv) {                               // Q heads
        if constexpr (TURN) {
            const int h0 = (role - 2 * c.nkv) * Q_HEADS, heads = min(Q_HEADS, a.nq - h0);
            const Weights g = weights_of(a.q_gamma);
            for (int t = from + row; t < to; t += ROWS) {
                const float *src = a.q + (w.row0 + t) * a.stride + (int64_t)h0 * c.hd;
                float *dst = a.qo + (w.row0 + t) * a.qo_stride + (int64_t)h0 * c.hd + ch;
                float y[Q_HEADS][4] = {}, z[Q_HEADS][4] = {}, fy[4], fz[4];
                factors_of(t, g, fy, fz);
#pragma unroll
                for (int h = 0; h < Q_HEADS; ++h)
                    if (h < heads) {
                        load(src + h * c.hd, y[h]);
                        load_other(src + h * c.hd, z[h]);
                    }
#pragma unroll
                for (int h = 0; h < Q_HEADS; ++h)
                    if (h < heads) {
                        float r[4];
                        turned(y[h], z[h], a.q_gamma != nullptr, fy, fz, r);
                        if (in)                           // (written past the L2: 84.7 -> 81.9 us)
                            __builtin_nontemporal_store(af4{r[0], r[1], r[2], r[3]},
                                                        reinterpret_cast<af4 *>(dst + h * c.hd));
                    }
            }
        }
        return;
    }

    const bool is_v = role >= c.nkv;
    const int page = append_page(c, w), h = is_v ? role - c.nkv : role;
    if (page < 0) {
        if (tid == 0 && role == 0)
            atomicOr(c.err, 1u);
        return;
    }
    const int slot = (int)(w.t0 & ((1 << c.ps_log2) - 1));
    const int64_t base = (int64_t)page * c.page_stride + (int64_t)h * c.block;
    const int64_t codes = (int64_t)c.hd << c.ps_log2;      // elements before an 8-bit block's scales

    if (!is_v) {                                           // K: a row's codes lie side by side
        const Weights g = weights_of(TURN ? a.k_gamma : nullptr);
        for (int t = from + row; t < to; t += ROWS) {
            const float *src = a.k + (w.row0 + t) * a.stride + (int64_t)h * c.hd;
            float y[4] = {};
            RK x[4];
            load(src, y);
            if constexpr (TURN) {
                float z[4] = {};
                RK fy[4], fz[4];
                load_other(src, z);
                factors_of(t, g, fy, fz);
                turned(y, z, a.k_gamma != nullptr, fy, fz, x);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x[e] = y[e];
            }
            const int64_t at = base + (int64_t)(slot + t) * c.hd + ch;
            if constexpr (SIZE == 1) {
                const float d = scale_of<T>(largest_of<LPR>(x));
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
        return;
    }

    // V: by rows into LDS, by channels out of it
    for (int t = from + row; t < to; t += ROWS) {
        float x[4] = {};
        load(a.v + (w.row0 + t) * a.stride + (int64_t)h * c.hd, x);
        if constexpr (SIZE == 1) {
            const float d = scale_of<T>(largest_of<LPR>(x));
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
static void launch_block(const QkvArgs &a, hipStream_t s)
{
    const bool vec = a.half % 4 == 0;
    const int64_t blocks = a.c.q_start ? (a.c.n_rows >> BL) + 2 * (int64_t)a.c.n_seq : a.c.n_seq;
    QkvArgs b = a;
    b.roles = 2 * a.c.nkv + (TURN ? (a.nq + Q_HEADS - 1) / Q_HEADS : 0);
    void (*k)(QkvArgs) = nullptr;
#define QG_APPEND_L(L) k = !TURN || vec ? k_qkv_append<T, BL, L, TURN, true> : k_qkv_append<T, BL, L, TURN, !TURN>
    switch (lanes_per_row(a.c.hd)) {
    case 16: QG_APPEND_L(16); break;
    case 32: QG_APPEND_L(32); break;
    default: QG_APPEND_L(64); break;
    }
#undef QG_APPEND_L
    // (a grid's row holds fewer than 2^32 threads; ids behind the last find no block)
    const int64_t all = blocks * b.roles, most = 1 << 23;
    const dim3 grid((unsigned)(all < most ? all : most), (unsigned)((all + most - 1) / most));
    hipLaunchKernelGGL(k, grid, dim3(256), 0, s, b);
}

template <int T, bool TURN>
static void launch_type(const QkvArgs &a, hipStream_t s)
{
    if (a.c.ps_log2 == 4)
        launch_block<T, 4, TURN>(a, s);
    else
        launch_block<T, 5, TURN>(a, s);
}

int launch_qkv_append(int kv_type, bool turn, const QkvArgs &a, void *stream)
{
    hipStream_t s = static_cast<hipStream_t>(stream);
    switch (kv_type) {
    case KV_I8: turn ? launch_type<KV_I8, true>(a, s) : launch_type<KV_I8, false>(a, s); break;
    case KV_F8: turn ? launch_type<KV_F8, true>(a, s) : launch_type<KV_F8, false>(a, s); break;
    case KV_F16: launch_type<KV_F16, true>(a, s); break;
    default: launch_type<KV_BF16, true>(a, s); break;
    }
    return (int)hipGetLastError();
}

}  // namespace qg
