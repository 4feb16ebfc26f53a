// attn_impl.h -- attention of one or a few new rows per sequence over f16 and bf16 pages.
//
// o = sum_t softmax(scale q . K_t) V_t for the query heads of one KV head: a workgroup takes up to
// 16 columns rho = token * group + head of them (one token: its heads) against one run (chunk) of
// positions.  Both products run on the matrix cores with the positions in the rows and the query
// heads in the columns, S^T = K Q^T and O^T = V^T P^T
// (v_mfma_f32_16x16x32), so that
//  - K, and V as the cache holds it (transposed inside the page), are the A operands: eight
//    consecutive halves each, loaded from the cache straight into registers by 16-byte loads;
//  - a lane's scores all belong to one query head (column l % 16), its running exponent, sum and
//    factors are per-lane scalars, and the scores it holds are exactly the probabilities it must
//    supply to the second product: row i of score tile tt is position 8 (i / 4) + 4 tt + i % 4 of a
//    32-position step, so lane group g = l / 16 holds positions 8 g .. 8 g + 7.
// The queries (times scale log2 e) and the probabilities are split into two or three f16 / bf16
// pieces whose products add up in f32 (PIECES); the matrix cores are idle otherwise.
//
// Each of the four waves takes every fourth 32-position step, loads one step ahead (K, V) and two
// ahead (page numbers), and keeps its own exponent, sum and O^T; they are joined in LDS at the end.
// The exponentials' reference (shift_of) moves by a wave vote, so the accumulators are hardly ever rescaled.
//
// Split over the length: the lengths are on the device, so every workgroup derives the same plan
// from them: the smallest chunk (whole 128-position units) for which the chunks of all sequences
// fit the grid's workgroup slots (where the sequences alone fill them, only the longest are split); a
// sequence's chunks are equal to one unit.  One chunk: the
// workgroup writes o.  Several: partial O, exponent and sum go to the workspace, and of every
// JOIN_RADIX chunks the last to finish adds them up (then of as many such groups, until one is
// left), always in chunk order, so that results do not depend on the order of execution.  A second
// launch for the joining took 4.5 us on the device and 3 us on the host of calls of 7 to 100 us.
//
// Bound by HBM where the cache is long: 64 sequences of 7500 positions (12 / 2 heads of 128, bf16) take
// 98 us, 5.04 TB/s; seven of up to 60000 (32 / 8, f16) 72 us, 5.16 TB/s.  By latency where it is short:
// 165 positions 6.8 us, one after the other the lengths, the page numbers, K and V.
#pragma once

#include "attn_shared.h"

namespace qg {

constexpr int JOIN_RADIX = 8;
// 16 columns; chunks of whole 128-position units, at least two; sequences of up to four are not split,
// and those of up to 32 not into more chunks than one join takes: four sequences of 4090 positions (32 / 8
// heads of 128) took 18.2 us with sixteen chunks and a second join, 15.9 with eight; one of 4090 (12 / 2)
// 10.9 and 11.2, and one of 5100 already 11.0 and 13.0.
template <bool SIDE> using AttnPlanOf = PlanOf<16, 7, 2, 4, 32, JOIN_RADIX, false, SIDE>;
typedef AttnPlanOf<false> AttnCols;

// LDS of a workgroup.
template <int T, int D>
struct AttnLds {
    // queries of the wide heads: every wave multiplies by the same ones, and in registers they would leave
    // none for the loads ahead
    static constexpr bool Q_LDS = D > 128;
    __attribute__((aligned(16))) float o[4][16][D];
    __attribute__((aligned(16))) au4 q[Q_LDS ? PIECES<T> * (D / 32) * 64 : 1];
    float m[4][16], l[4][16], mo[16], lo[16];
    int last, done[16];
};

// Partial results of a slot: the tile's O (unnormalised) [cols][hd], then (exponent, sum) [cols].
// SIDE: several tiles of a KV head read the same positions.  They come next to each other and on one XCD
// (workgroups eight apart), so that one of them finds the other's in the L2: 64 sequences of 7500 positions,
// 40 / 2 heads of 128: 140.9 us tile by tile, 107 to 111; of 64 75.0 and 58; sixteen of 8 rows x 4000, 24 / 2:
// 53.3 and 47.6.  (In the code of the others it costs 0.15 of 7 us.)
template <int T, int D, int FORM, bool SIDE>
__device__ __forceinline__ void attn_body(const AttnArgs &a, int slots, int id, int grid, AttnLds<T, D> &sh)
{
    constexpr bool ROWS = FORM == MANY || FORM == PREFIX;
    constexpr int KB = D / 32, DT = D / 16, NP = PIECES<T>;
    constexpr bool Q_LDS = AttnLds<T, D>::Q_LDS;
    const KvArgs &c = a.c;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int i = lane & 15, g = lane >> 4;
    AttnPlan p;
    if constexpr (SIDE) {
        const int run = 8 * a.side, r = id % run;
        if (id - r + run <= grid)
            id += r % 8 * a.side + r / 8 - r;
    }
    if (!attn_plan<AttnPlanOf<SIDE>, FORM>(a, slots, id, p, reinterpret_cast<AttnSeq *>(&sh.o[0][0][0])))
        return;
    // (PREFIX: a group's first sequence, whose pages are read)
    const int b = FORM == PREFIX ? p.row0 : p.b, chunk = p.chunk, n_chunk = p.n_chunk;
    // behind a prefix: the shared positions are in the pages of another, the plan's begin at base
    const int shared = behind(FORM) && p.sound ? shared_of(a, b) : 0, base = behind(FORM) ? suffix_base(shared) : 0;
    int len = behind(FORM) && p.len > 0 ? base + p.len : p.len;
    const int tiles = (p.rows * a.group + 15) / 16, hkv = p.pair / tiles, rho0 = p.pair % tiles * 16;
    const int cols = min(16, p.rows * a.group - rho0);
    // offset of column col in o, and of its row and head in q
    auto head_of = [&](int col) { return hkv * a.group + (ROWS ? (rho0 + col) % a.group : rho0 + col); };
    auto row_of = [&](int col) { return p.row0 + (ROWS ? (rho0 + col) / a.group : 0); };

    // this chunk's 32-position steps, dealt to the waves in turn
    const int units = AttnCols::units(p.len);
    const int per = units / n_chunk, more = units % n_chunk;
    const int unit0 = chunk * per + min(chunk, more);
    const int t_begin = base + (unit0 << AttnCols::UNIT_LOG2);
    int t_end = min(len, base + ((unit0 + per + (chunk < more ? 1 : 0)) << AttnCols::UNIT_LOG2));
    // positions this lane's column sees, [0, see), and those that all columns see (columns without a
    // row see what the last one does and are not stored)
    int see = t_end, see_all = t_end;
    if constexpr (FORM == PREFIX) {
        see = min(t_end, prefix_seen(a, row_of(min(i, cols - 1)), len));
    } else if constexpr (FORM == MANY) {
        const int pos0 = max(c.kv_len[b], -(1 << 30)) - p.rows;
        see = min(t_end, pos0 + (rho0 + min(i, cols - 1)) / a.group + 1);
        see_all = min(t_end, pos0 + rho0 / a.group + 1);
    }

    // queries of column i: scaled, split
    au4 qf[Q_LDS ? 1 : NP][Q_LDS ? 1 : KB];
    float unscale;
    {
        const int col = i < cols ? i : 0;
        const float *qr = a.q + (int64_t)row_of(col) * a.q_stride + (int64_t)head_of(col) * D;
        float v[KB][8], amax = 0.f;
        const float f = i < cols ? a.scale * LOG2E : 0.f;
#pragma unroll
        for (int k = 0; k < KB; ++k) {
            const float4 x = *reinterpret_cast<const float4 *>(qr + 32 * k + 8 * g);
            const float4 y = *reinterpret_cast<const float4 *>(qr + 32 * k + 8 * g + 4);
            const float w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[k][e] = i < cols ? w[e] : 0.f;
                amax = fmaxf(amax, fabsf(v[k][e]));
            }
        }
        const float sc = q_scale<T>(max_x32(max_x16(amax)));
        unscale = f / sc;
#pragma unroll
        for (int k = 0; k < KB; ++k) {
            float w[8];
            au4 out[NP];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                w[e] = v[k][e] * sc;
            split8<T>(w, out);
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
    const int n_steps = t_end > t_begin + 32 * wave ? (t_end - t_begin - 32 * wave + 127) / 128 : 0;
    if constexpr (Q_LDS)
        __syncthreads();

    af4 o[DT];
#pragma unroll
    for (int d = 0; d < DT; ++d)
        o[d] = af4{0.f, 0.f, 0.f, 0.f};
    float shift = NO_SHIFT, l = 0.f;

    if (n_steps > 0) {
        const int last_entry = (len - 1) >> c.ps_log2, ps_mask = (1 << c.ps_log2) - 1;
        const int32_t *table = c.table + (int64_t)b * c.max_pages;
        const int64_t head = (int64_t)hkv * D << c.ps_log2;
        const int tok_k = 8 * (i >> 2) + (i & 3);         // + 4 tt: position of K row i in a step
        const int64_t np = c.n_pages;
        struct Ids {
            int k, v;
        };
        struct Buf {
            au4 k[2][KB], v[DT];
            bool bad;                                     // this lane's positions have no page
        };
        auto step_t = [&](int s) { return t_begin + 32 * wave + 128 * (s < n_steps ? s : n_steps - 1); };
        auto ids_of = [&](int s) {
            const int t = step_t(s);
            Ids r;
            r.k = table[min((t + tok_k) >> c.ps_log2, last_entry)];
            r.v = table[min((t + 8 * g) >> c.ps_log2, last_entry)];
            return r;
        };
        auto issue = [&](Buf &x, int s, const Ids &id) {
            const int t = step_t(s);
            const bool okk = id.k >= 0 && id.k < np, okv = id.v >= 0 && id.v < np;
            x.bad = !okv;
            const uint16_t *kp = c.k + ((okk ? (int64_t)id.k : 0) * c.page_stride + head) + 8 * g;
            const uint16_t *vp = c.v + ((okv ? (int64_t)id.v : 0) * c.page_stride + head) +
                                 (i << c.ps_log2) + ((t + 8 * g) & ps_mask);
#pragma unroll
            for (int tt = 0; tt < 2; ++tt)
#pragma unroll
                for (int k = 0; k < KB; ++k)
                    x.k[tt][k] = *reinterpret_cast<const au4 *>(kp + ((t + tok_k + 4 * tt) & ps_mask) * D + 32 * k);
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
            float sc[8];
#pragma unroll
            for (int tt = 0; tt < 2; ++tt) {
                af4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int y = NP - 1; y >= 0; --y)
#pragma unroll
                    for (int k = 0; k < KB; ++k)
                        acc = mm16<T>(x.k[tt][k], q_at(y, k), acc);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    sc[4 * tt + r] = acc[r] * unscale;
            }
            const uint64_t any_bad = __ballot(x.bad);
            bool odd = false;
            uint16_t *sv = reinterpret_cast<uint16_t *>(&sh.o[wave][0][0]);      // [D][32]
            if (any_bad != 0 || t + 32 > see_all || (behind(FORM) && t < shared)) {
                if (any_bad && lane == 0)
                    atomicOr(c.err, 1u);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    sc[e] = x.bad || t + 8 * g + e >= see || (behind(FORM) && t + 8 * g + e < shared) ? -INFINITY
                                                                                               : sc[e];
                // what a masked position holds must not reach the product: 0 x NaN is NaN
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const int tw = t + 8 * g + 2 * w;
                    uint32_t keep = x.bad || tw >= t_end ? 0u : tw + 1 >= t_end ? 0xFFFFu : ~0u;
                    if constexpr (behind(FORM))
                        keep &= tw + 1 < shared ? 0u : tw < shared ? 0xFFFF0000u : ~0u;
#pragma unroll
                    for (int d = 0; d < DT; ++d)
                        x.v[d][w] &= keep;
                }
                // positions that some columns see: infinities and NaN leave the product and are
                // added one by one to the columns that see them
                if constexpr (ROWS) {
                    uint32_t nf = 0;
#pragma unroll
                    for (int d = 0; d < DT; ++d)
#pragma unroll
                        for (int w = 0; w < 4; ++w)
                            nf |= nonfinite2<T>(x.v[d][w]);
                    odd = __any(nf != 0);
                    if (odd) {
#pragma unroll
                        for (int d = 0; d < DT; ++d) {
                            *reinterpret_cast<au4 *>(sv + (16 * d + i) * 32 + 8 * g) = x.v[d];
#pragma unroll
                            for (int w = 0; w < 4; ++w) {
                                const uint32_t f = nonfinite2<T>(x.v[d][w]);
                                x.v[d][w] &= ~((f - (f >> 15)) | f);
                            }
                        }
                        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
                        __builtin_amdgcn_wave_barrier();
                        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
                    }
                }
            }
            float mx = fmaxf(fmaxf(fmaxf(sc[0], sc[1]), fmaxf(sc[2], sc[3])),
                             fmaxf(fmaxf(sc[4], sc[5]), fmaxf(sc[6], sc[7])));
            if (__any(mx + shift > TOP<T>)) {
                const float to = fminf(shift, shift_of<T>(max_x32(max_x16(mx))));
                const float f = __builtin_amdgcn_exp2f(to - shift);
                shift = to;
                l *= f;
#pragma unroll
                for (int d = 0; d < DT; ++d)
                    o[d] *= f;
            }
            float pr[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                pr[e] = __builtin_amdgcn_exp2f(sc[e] + shift);
                l += pr[e];
            }
            au4 pf[NP];
            split8<T>(pr, pf);
#pragma unroll
            for (int y = NP - 1; y >= 0; --y)
#pragma unroll
                for (int d = 0; d < DT; ++d)
                    o[d] = mm16<T>(x.v[d], pf[y], o[d]);
            if (ROWS && odd) {
#pragma unroll 1
                for (int y = 0; y < 32 && t + y < t_end; ++y)
#pragma unroll
                    for (int d = 0; d < DT; ++d)
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const uint32_t v = sv[(16 * d + 4 * g + r) * 32 + y];
                            if (t + y < see && nonfinite2<T>(v))
                                o[d][r] += low_of<T>(v);
                            if (r == 3)
                                __builtin_amdgcn_sched_barrier(0);
                        }
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

    // join the waves: column i of O^T, rows 16 d + 4 g + r
    l = sum_x32(sum_x16(l));
    if (g == 0) {
        sh.m[wave][i] = -shift;
        sh.l[wave][i] = l;
    }
#pragma unroll
    for (int d = 0; d < DT; ++d)
        *reinterpret_cast<af4 *>(&sh.o[wave][i][16 * d + 4 * g]) = o[d];
    __syncthreads();
    const int width = ROWS ? 16 : min(16, a.group), items = cols * (D / 4);
    const uint32_t stride = (uint32_t)attn_part_floats(width, D);
    const __amdgpu_buffer_rsrc_t part = __builtin_amdgcn_make_buffer_rsrc(
        (behind(FORM) ? a.tail_part : a.part) + (int64_t)p.slot0 * stride, 0, n_chunk * stride * 4, 0x00020000);
    // four channels of a column to o, or to where the halves meet
    auto store = [&](int e, af4 sum, float m, float ls) {
        const af4 mean = sum * inverse_sum(ls);
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
        const float mm = fmaxf(fmaxf(sh.m[0][col], sh.m[1][col]), fmaxf(sh.m[2][col], sh.m[3][col]));
        af4 sum = {0.f, 0.f, 0.f, 0.f};
        float ls = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float f = join_weight(sh.m[w][col], mm);
            sum += *reinterpret_cast<const af4 *>(&sh.o[w][col][4 * d4]) * f;
            ls += sh.l[w][col] * f;
        }
        if (n_chunk == 1) {
            store(e, sum, mm, ls);
        } else {
            put4(part, part_at(chunk, e), sum);
            if (d4 == 0)
                put2(part, sums_at(chunk, col), mm, ls);
        }
    }
    if (n_chunk == 1) {
        finish();
        return;
    }
    // nodes of 1, 8, 64, ... chunks; a node's result lies in the slot of its first chunk.  The group
    // that starts at chunk g0 of level L arrives at the pair's counter g0 + L: all of a level's g0
    // are multiples of JOIN_RADIX, so no two share one
    for (int node = 1, level = 0; node < n_chunk; node *= JOIN_RADIX, ++level) {
        const int g0 = chunk / (node * JOIN_RADIX) * (node * JOIN_RADIX);
        const int members = min(JOIN_RADIX, (n_chunk - g0 + node - 1) / node);
        if (members == 1)
            continue;                                     // already in its place
        if (!last_to_arrive((behind(FORM) ? a.tail_count : a.count) + p.slot0 + g0 + level, members, &sh.last))
            return;
        const bool top = node * JOIN_RADIX >= n_chunk;
        for (int e = threadIdx.x; e < items; e += 256) {
            const int col = e / (D / 4), d4 = e % (D / 4);
            float mk[JOIN_RADIX], lk[JOIN_RADIX];
            af4 x[JOIN_RADIX];
#pragma unroll
            for (int k = 0; k < JOIN_RADIX; ++k) {              // all loads in flight at once
                mk[k] = -INFINITY;
                if (k < members) {
                    get2(part, sums_at(g0 + k * node, col), mk[k], lk[k]);
                    x[k] = get4(part, part_at(g0 + k * node, e));
                }
            }
            float mm = -INFINITY, ls = 0.f;
#pragma unroll
            for (int k = 0; k < JOIN_RADIX; ++k)
                mm = fmaxf(mm, mk[k]);
            af4 sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < JOIN_RADIX; ++k)
                if (k < members) {
                    const float f = join_weight(mk[k], mm);
                    sum += x[k] * f;
                    ls += lk[k] * f;
                }
            if (top) {
                store(e, sum, mm, ls);
            } else {
                // the exponent and sum replace what other threads of the column may still have to read
                put4(part, part_at(g0, e), sum);
                if (d4 == 0) {
                    sh.mo[col] = mm;
                    sh.lo[col] = ls;
                }
            }
        }
        if (top) {
            finish();
        } else {
            __syncthreads();
            if ((int)threadIdx.x < cols)
                put2(part, sums_at(g0, threadIdx.x), sh.mo[threadIdx.x], sh.lo[threadIdx.x]);
        }
    }
}

}  // namespace qg
