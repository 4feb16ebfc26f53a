// attn8_impl.h -- attention of one or a few new rows per sequence over 8-bit pages.
//
// As over f16 pages (attn_impl.h): a workgroup takes up to 16 columns rho = token * group + head of a KV
// head against a chunk of positions, S^T = K Q^T and O^T = V^T P^T on v_mfma_f32_16x16x32_f16, the plan from the
// lengths on the device, parts joined in the launch.  What the bytes change:
//  - a step of a wave is 64 positions, so that a lane's loads stay 16 bytes: of K sixteen channels of a position
//    (two operands, queries in the same order), of V^T sixteen positions of a channel.  Row i of score tile tt is
//    position 16 (i / 4) + 4 tt + i % 4, so lane group g holds the scores of positions 16 g .. 16 g + 15, which its
//    V operands want;
//  - lane i of group g loads the scales of position 16 g + i, and a score takes its own by a lane broadcast within
//    16 lanes (one instruction's operand);
//  - parts are means (attn_bytes.h).
//
// Bound by HBM with long caches: 64 tokens over ~7500 positions each, 24 / 8 heads of 64, I8 (524 MB), 105 us, 5.0
// TB/s (f16 pages: 1.9 times the bytes); seven, the longest of 60000 positions, 32 / 8 heads of 128, F8 (191 MB),
// 43 us.  One token over 180 positions 6.6 us, latency.  The conversion of the codes, 2 to 2.5 vector instructions
// for four, hides behind the loads.
#pragma once

#include "attn_bytes.h"
#include "attn_shared.h"

namespace qg {

constexpr int JOIN8_RADIX = 8;
template <bool SIDE> using Attn8PlanOf = PlanOf<16, 8, 1, 2, 16, JOIN8_RADIX, false, SIDE>;
typedef Attn8PlanOf<false> Attn8Cols;

// LDS of a workgroup.
template <int T, int D>
struct Attn8Lds {
    // queries of the wide heads: every wave multiplies by the same ones, and in registers they would leave
    // none for the loads ahead
    static constexpr bool Q_LDS = D > 128;
    __attribute__((aligned(16))) float o[4][16][D];
    __attribute__((aligned(16))) au4 q[Q_LDS ? 2 * (D / 32) * 64 : 1];
    float m[4][16], l[4][16];
    int last, done[16];
};

template <int T, int D, int FORM, bool SIDE>
__device__ __forceinline__ void attn8_body(const AttnArgs &a, int slots, int id, int grid, Attn8Lds<T, D> &sh)
{
    constexpr bool ROWS = FORM == MANY || FORM == PREFIX;
    constexpr int KB = D / 32, DT = D / 16, NP = 2, KP = D / 64, REST = D % 64 / 32;
    constexpr bool Q_LDS = Attn8Lds<T, D>::Q_LDS;
    const KvArgs &c = a.c;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int i = lane & 15, g = lane >> 4;
    AttnPlan p;
    if constexpr (SIDE) {
        const int run = 8 * a.side, r = id % run;
        if (id - r + run <= grid)
            id += r % 8 * a.side + r / 8 - r;
    }
    if (!attn_plan<Attn8PlanOf<SIDE>, FORM>(a, slots, id, p, reinterpret_cast<AttnSeq *>(&sh.o[0][0][0])))
        return;
    // (PREFIX: a group's first sequence, whose pages are read)
    const int b = FORM == PREFIX ? p.row0 : p.b, chunk = p.chunk, n_chunk = p.n_chunk;
    // behind a prefix: the shared positions are in the pages of another, the plan's begin at base
    const int shared = behind(FORM) && p.sound ? shared_of(a, b) : 0, base = behind(FORM) ? suffix_base(shared) : 0;
    int len = behind(FORM) && p.len > 0 ? base + p.len : p.len;
    const int tiles = (p.rows * a.group + 15) / 16, hkv = p.pair / tiles, rho0 = p.pair % tiles * 16;
    const int cols = min(16, p.rows * a.group - rho0);
    auto head_of = [&](int col) { return hkv * a.group + (ROWS ? (rho0 + col) % a.group : rho0 + col); };
    auto row_of = [&](int col) { return p.row0 + (ROWS ? (rho0 + col) / a.group : 0); };

    // this chunk's 64-position steps, dealt to the waves in turn
    const int units = Attn8Cols::units(p.len);
    const int per = units / n_chunk, more = units % n_chunk;
    const int unit0 = chunk * per + min(chunk, more);
    const int t_begin = base + (unit0 << Attn8Cols::UNIT_LOG2);
    int t_end = min(len, base + ((unit0 + per + (chunk < more ? 1 : 0)) << Attn8Cols::UNIT_LOG2));
    // positions this lane's column sees, [0, see), and those that all columns see
    int see = t_end, see_all = t_end;
    if constexpr (FORM == PREFIX) {
        see = min(t_end, prefix_seen(a, row_of(min(i, cols - 1)), len));
    } else if constexpr (FORM == MANY) {
        const int pos0 = max(c.kv_len[b], -(1 << 30)) - p.rows;
        see = min(t_end, pos0 + (rho0 + min(i, cols - 1)) / a.group + 1);
        see_all = min(t_end, pos0 + rho0 / a.group + 1);
    }

    // queries of column i: scaled, split, in the order of the channels in K's operands
    auto channel = [&](int k) { return k < 2 * KP ? 64 * (k >> 1) + 16 * g + 8 * (k & 1) : 64 * KP + 8 * g; };
    au4 qf[Q_LDS ? 1 : NP][Q_LDS ? 1 : KB];
    // a score is (product * unscale) * d^K * lift: lift, a power of two from 1 on, takes what queries near f32's
    // end would make of the first product, which K's scale may bring down again
    float unscale, lift = 1.0f;
    {
        const int col = i < cols ? i : 0;
        const float *qr = a.q + (int64_t)row_of(col) * a.q_stride + (int64_t)head_of(col) * D;
        float v[KB][8], amax = 0.f;
        const float f = i < cols ? a.scale * LOG2E : 0.f;
#pragma unroll
        for (int k = 0; k < KB; ++k) {
            const float4 x = *reinterpret_cast<const float4 *>(qr + channel(k));
            const float4 y = *reinterpret_cast<const float4 *>(qr + channel(k) + 4);
            const float w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[k][e] = i < cols ? w[e] : 0.f;
                amax = fmaxf(amax, fabsf(v[k][e]));
            }
        }
        const float sc = q_scale<KV_F16>(max_x32(max_x16(amax)));
        unscale = f / sc;
        int e2 = 0;
        frexpf(unscale, &e2);
        if (e2 > 0) {
            lift = ldexpf(1.0f, e2);
            unscale = ldexpf(unscale, -e2);
        }
#pragma unroll
        for (int k = 0; k < KB; ++k) {
            float w[8];
            au4 out[NP];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                w[e] = v[k][e] * sc;
            split8<KV_F16>(w, out);
#pragma unroll
            for (int x = 0; x < NP; ++x)
                if constexpr (!Q_LDS)
                    qf[x][k] = out[x];
                else if (k % 4 == wave)
                    sh.q[(x * KB + k) * 64 + lane] = out[x];
        }
    }
    if constexpr (FORM == PREFIX) {
        // what none of these rows sees is not read (positions are below 2^24, whole numbers in f32); the rows' lengths
        // have arrived by now
        t_end = __builtin_amdgcn_readfirstlane((int)max_of_16((float)see));
        len = min(len, t_end);
        see_all = -(int)max_of_16(-(float)see);
    }
    const int n_steps = t_end > t_begin + 64 * wave ? (t_end - t_begin - 64 * wave + 255) / 256 : 0;
    if constexpr (Q_LDS)
        __syncthreads();

    af4 o[DT];
#pragma unroll
    for (int d = 0; d < DT; ++d)
        o[d] = af4{0.f, 0.f, 0.f, 0.f};
    // r: the wave's reference of V's scales; top: the column's largest scale above it
    float shift = NO_SHIFT, l = 0.f, r = -200.0f, top = LEAST_TOP;

    if (n_steps > 0) {
        const int last_entry = (len - 1) >> c.ps_log2, ps_mask = (1 << c.ps_log2) - 1;
        const int32_t *table = c.table + (int64_t)b * c.max_pages;
        const int64_t head = (int64_t)hkv * c.block, scales = (int64_t)D << c.ps_log2;
        const int64_t np = c.n_pages;
        struct Ids {
            int k, v;
        };
        struct Buf {
            au4 k[4][KP], v[DT];
            uint2 kr[4][REST ? 1 : 0];
            float dk, dv;                                 // scales of position 16 g + i
            bool bad;                                     // positions 16 g .. 16 g + 15 have no page
        };
        auto step_t = [&](int s) { return t_begin + 64 * wave + 256 * (s < n_steps ? s : n_steps - 1); };
        // K row i of a tile lies in 16-position block i / 4, V and the scales in block g
        auto ids_of = [&](int s) {
            const int t = step_t(s);
            Ids x;
            x.k = table[min((t + 16 * (i >> 2)) >> c.ps_log2, last_entry)];
            x.v = table[min((t + 16 * g) >> c.ps_log2, last_entry)];
            return x;
        };
        auto issue = [&](Buf &x, int s, const Ids &id) {
            const int t = step_t(s);
            const bool okk = id.k >= 0 && id.k < np, okv = id.v >= 0 && id.v < np;
            x.bad = !okv;
            const int tk = t + 16 * (i >> 2) + (i & 3), tv = t + 16 * g;
            const uint8_t *kp = c.k8() + ((okk ? (int64_t)id.k : 0) * c.page_stride + head) + (tk & ps_mask) * D;
            const int64_t at = (okv ? (int64_t)id.v : 0) * c.page_stride + head;
            const uint8_t *vp = c.v8() + at + (i << c.ps_log2) + (tv & ps_mask);
            const int64_t ds = at + scales + 4 * ((tv & ps_mask) + i);
            x.dk = *reinterpret_cast<const float *>(c.k8() + ds);
            x.dv = *reinterpret_cast<const float *>(c.v8() + ds);
#pragma unroll
            for (int tt = 0; tt < 4; ++tt) {
#pragma unroll
                for (int k = 0; k < KP; ++k)
                    x.k[tt][k] = *reinterpret_cast<const au4 *>(kp + 4 * tt * D + 64 * k + 16 * g);
                if constexpr (REST)
                    x.kr[tt][0] = *reinterpret_cast<const uint2 *>(kp + 4 * tt * D + 64 * KP + 8 * g);
            }
#pragma unroll
            for (int d = 0; d < DT; ++d)
                x.v[d] = *reinterpret_cast<const au4 *>(vp + ((16 * d) << c.ps_log2));
        };
        auto q_at = [&](int y, int k) {
            if constexpr (Q_LDS)
                return sh.q[(y * KB + k) * 64 + lane];
            else
                return qf[y][k];
        };
        auto compute = [&](Buf &x, int s) {
            const int t = step_t(s);
            if constexpr (Q_LDS)
                asm volatile("" ::: "memory");            // the queries are read anew each step
            float sc[16];
#pragma unroll
            for (int tt = 0; tt < 4; ++tt) {
                af4 acc[NP];
#pragma unroll
                for (int y = 0; y < NP; ++y)
                    acc[y] = af4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int k = 0; k < KP; ++k) {
                    au4 lo, hi;
                    halves_of<T>(x.k[tt][k], lo, hi);
#pragma unroll
                    for (int y = 0; y < NP; ++y)
                        acc[y] = mm16<KV_F16>(hi, q_at(y, 2 * k + 1), mm16<KV_F16>(lo, q_at(y, 2 * k), acc[y]));
                }
                if constexpr (REST) {
                    au4 lo, hi;
                    halves_of<T>(au4{x.kr[tt][0].x, x.kr[tt][0].y, 0u, 0u}, lo, hi);
#pragma unroll
                    for (int y = 0; y < NP; ++y)
                        acc[y] = mm16<KV_F16>(lo, q_at(y, 2 * KP), acc[y]);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    sc[4 * tt + e] = (acc[1][e] + acc[0][e]) * unscale;
            }
            times_lanes([&](int e) -> float & { return sc[e]; }, x.dk);
            const uint64_t any_bad = __ballot(x.bad);
            const bool edge = any_bad != 0 || t + 64 > see_all || (behind(FORM) && t < shared);
            uint32_t hide = 0;                            // of this column's 16 positions
            float dv = x.dv;
            if (edge) {
                if (any_bad && lane == 0)
                    atomicOr(c.err, 1u);
                const int n = x.bad ? 0 : see - t - 16 * g;
                hide = n >= 16 ? 0u : n <= 0 ? 0xFFFFu : 0xFFFFu & (0xFFFFu << n);
                const int skip = behind(FORM) ? shared - t - 16 * g : 0;        // < 16
                if (behind(FORM) && skip > 0)
                    hide |= (1u << skip) - 1u;
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    sc[e] = hide >> e & 1 ? -INFINITY : sc[e];
                const int left = x.bad ? 0 : t_end - t - 16 * g;      // positions of the group that exist
                dv = i < left && (!behind(FORM) || i >= skip) ? dv : 0.f;
                // what a masked position holds must not reach the product: an e4m3 may be NaN
                if constexpr (T == KV_F8)
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const int m = left - 4 * w;
                        uint32_t keep = m >= 4 ? ~0u : m <= 0 ? 0u : (1u << (8 * m)) - 1u;
                        if constexpr (behind(FORM)) {
                            const int k = skip - 4 * w;
                            keep &= k >= 4 ? 0u : k <= 0 ? ~0u : ~0u << (8 * k);
                        }
#pragma unroll
                        for (int d = 0; d < DT; ++d)
                            x.v[d][w] &= keep;
                    }
            }
            // scales: relative to 2^r; the largest that the column sees
            float seen = dv;
            if (ROWS && edge) {
                seen = 0.f;
                each_lane([&](int e, float v) { seen = hide >> e & 1 ? seen : fmaxf(seen, v); }, dv);
                seen = max_x32(max_x16(seen));
            } else {
                seen = max_x32(max_x16(max_of_16(seen)));
            }
            const float most = ROWS && edge ? max_of_16(exponent_above(seen)) : exponent_above(seen);
            top = fmaxf(top, exponent_above(seen) - r);
            float mx = sc[0];
#pragma unroll
            for (int e = 1; e < 16; ++e)
                mx = fmaxf(mx, sc[e]);
            mx *= lift;
            const bool moved = __builtin_amdgcn_readfirstlane(most > r + R_SLACK);
            if (moved || __any(mx + shift > TOP8 - top)) {
                const float to = moved ? most : r;
                const Rescaled x = rescaled(r, to, top, shift, max_x32(max_x16(mx)), exponent_above(max_x32(max_x16(l))));
                r = to;
                top = x.top;
                shift = x.shift;
                l *= x.l;
#pragma unroll
                for (int d = 0; d < DT; ++d)
                    o[d] *= x.o;
            }
            dv = ldexpf(dv, -(int)r);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                sc[e] = __builtin_amdgcn_exp2f(fmaf(sc[e], lift, shift));
                l += sc[e];
            }
            times_lanes([&](int e) -> float & { return sc[e]; }, dv);
            if (ROWS && edge) {                           // a NaN scale that this column does not see
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    sc[e] = hide >> e & 1 ? 0.f : sc[e];
            }
            au4 pf[2][NP];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float w[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    w[e] = sc[8 * h + e];
                split8<KV_F16>(w, pf[h]);
            }
#pragma unroll
            for (int d = 0; d < DT; ++d) {
                au4 lo, hi;
                halves_of<T>(x.v[d], lo, hi);
#pragma unroll
                for (int y = NP - 1; y >= 0; --y)
                    o[d] = mm16<KV_F16>(hi, pf[1][y], mm16<KV_F16>(lo, pf[0][y], o[d]));
            }
        };
        Buf A, B;
        Ids i0 = ids_of(0), i1 = ids_of(1);
        issue(A, 0, i0);
        for (int s = 0; s < n_steps; s += 2) {
            i0 = ids_of(s + 2);
            issue(B, s + 1, i1);
            compute(A, s);
            i1 = ids_of(s + 3);
            issue(A, s + 2, i0);
            if (s + 1 < n_steps)
                compute(B, s + 1);
        }
    }

    // join the waves: column i of O^T, rows 16 d + 4 g + e
    l = sum_x32(sum_x16(l));
    if (g == 0) {
        sh.m[wave][i] = -shift;
        sh.l[wave][i] = l;
    }
    {
        const float f = inverse_sum(l);
#pragma unroll
        for (int d = 0; d < DT; ++d) {
            af4 v = o[d] * f;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[e] = ldexpf(v[e], (int)r);
            *reinterpret_cast<af4 *>(&sh.o[wave][i][16 * d + 4 * g]) = v;
        }
    }
    __syncthreads();
    const int width = ROWS ? 16 : min(16, a.group), items = cols * (D / 4);
    const uint32_t stride = (uint32_t)attn_part_floats(width, D);
    const __amdgpu_buffer_rsrc_t part = __builtin_amdgcn_make_buffer_rsrc(
        (behind(FORM) ? a.tail_part : a.part) + (int64_t)p.slot0 * stride, 0, n_chunk * stride * 4, 0x00020000);
    // four channels of a column to o, or to where the halves meet
    auto store = [&](int e, af4 mean, float m, float ls) {
        const int col = e / (D / 4), d4 = e % (D / 4);
        const int64_t at = (int64_t)row_of(col) * a.nq + head_of(col);
        if (FORM == PREFIX || (FORM == SUFFIX && shared > 0)) {
            meet_put<D>(a, FORM == PREFIX ? 0 : 1, at, d4, mean, m, ls);
            return;
        }
        *reinterpret_cast<af4 *>(a.o + at * D + 4 * d4) = mean;
        if (FORM == TAIL && d4 == 0)
            *reinterpret_cast<float2 *>(a.stats + 2 * at) = make_float2(m, ls);
    };
    // all of the columns are stored
    auto finish = [&]() {
        if constexpr (FORM == PREFIX) {
            const int m0 = rho0 / a.group, n = (rho0 + cols - 1) / a.group - m0 + 1;
            meet<D>(a, p.row0 + m0, n, hkv, sh.done,
                    [&](int i) { return shared_of(a, p.row0 + m0 + i) > 0 ? meeting(m0 + i, a.group) : 0; });
        } else if constexpr (FORM == SUFFIX) {
            if (shared > 0) {
                const int m = b - group_first(a, b);
                meet<D>(a, b, 1, hkv, sh.done, [&](int) { return meeting(m, a.group); });
            }
        }
    };
    auto sums_at = [&](int at, int col) { return at * stride + width * D + 2 * col; };
    auto part_at = [&](int at, int e) { return at * stride + 4 * e; };

    for (int e = threadIdx.x; e < items; e += 256) {
        const int col = e / (D / 4), d4 = e % (D / 4);
        const float m[4] = {sh.m[0][col], sh.m[1][col], sh.m[2][col], sh.m[3][col]};
        const float ls[4] = {sh.l[0][col], sh.l[1][col], sh.l[2][col], sh.l[3][col]};
        float f[4];
        const Factors j = join_factors(m, ls, 4, f);
        af4 mean = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < 4; ++w)
            mean += *reinterpret_cast<const af4 *>(&sh.o[w][col][4 * d4]) * f[w];
        if (n_chunk == 1) {
            store(e, mean, j.m, j.l);
        } else {
            put4(part, part_at(chunk, e), mean);
            if (d4 == 0)
                put2(part, sums_at(chunk, col), j.m, j.l);
        }
    }
    if (n_chunk == 1) {
        finish();
        return;
    }
    // nodes of 1, 8, 64, ... chunks, as over f16 pages
    for (int node = 1, level = 0; node < n_chunk; node *= JOIN8_RADIX, ++level) {
        const int g0 = chunk / (node * JOIN8_RADIX) * (node * JOIN8_RADIX);
        const int members = min(JOIN8_RADIX, (n_chunk - g0 + node - 1) / node);
        if (members == 1)
            continue;                                     // already in its place
        if (!last_to_arrive((behind(FORM) ? a.tail_count : a.count) + p.slot0 + g0 + level, members, &sh.last))
            return;
        const bool last = node * JOIN8_RADIX >= n_chunk;
        for (int e = threadIdx.x; e < items; e += 256) {
            const int col = e / (D / 4), d4 = e % (D / 4);
            float m[JOIN8_RADIX], ls[JOIN8_RADIX], f[JOIN8_RADIX];
            af4 x[JOIN8_RADIX];
#pragma unroll
            for (int k = 0; k < JOIN8_RADIX; ++k)         // all loads in flight at once
                if (k < members) {
                    get2(part, sums_at(g0 + k * node, col), m[k], ls[k]);
                    x[k] = get4(part, part_at(g0 + k * node, e));
                }
            const Factors j = join_factors(m, ls, members, f);
            af4 mean = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < JOIN8_RADIX; ++k)
                if (k < members)
                    mean += x[k] * f[k];
            if (last) {
                store(e, mean, j.m, j.l);
            } else {
                // the exponent and sum replace what other threads of the column may still have to read
                put4(part, part_at(g0, e), mean);
                if (d4 == 0) {
                    sh.m[0][col] = j.m;
                    sh.l[0][col] = j.l;
                }
            }
        }
        if (last) {
            finish();
        } else {
            __syncthreads();
            if ((int)threadIdx.x < cols)
                put2(part, sums_at(g0, threadIdx.x), sh.m[0][threadIdx.x], sh.l[0][threadIdx.x]);
        }
    }
}

}  // namespace qg
