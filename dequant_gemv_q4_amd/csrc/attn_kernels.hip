// attn_kernels.hip -- the paged key-value cache: storing new rows, and attention of one new token per
// sequence over it.
#include <hip/hip_runtime.h>

#include "attn_common.h"

namespace qg {

// ------------------------------------------------------------------------------------ new rows
//
// A workgroup stores one KV head of one block of 16 or 32 positions (at most a page) of a sequence.
// K: a thread takes eight channels of a position (32 bytes read, 16 written).  V is transposed on
// the way: a thread takes eight positions of a channel, one 4-byte load each, and writes them as 16
// bytes; neighbouring lanes take the pieces of a channel, then the next channel, so that a wave
// writes 1 KB in one run (pages of 16 and 32) or in runs of 64 bytes, and reads runs of 64 or 128
// bytes.  A piece with positions that are not new is written element by element.
//
// Blocks start at multiples of their size; sequence b's begin at block id q_start[b] / size + 2 b,
// which leaves every sequence enough ids wherever its first position lies.
//
// Bound by HBM: 8000 rows of 8 heads of 128 (98.3 MB read and written) take 22.4 us, 4.4 TB/s, where a
// copy reaches 4.94; one position at a time took 75 us.  One row of 2 heads: 2.8 us, a launch.
template <int T, int BL>
__global__ __launch_bounds__(256) void k_kv_append(AppendArgs a)
{
    constexpr int BLOCK = 1 << BL, PIECES_V = BLOCK / 8;
    const KvArgs &c = a.c;
    const int tid = threadIdx.x, lane = tid & 63, h = blockIdx.y;
    int id = blockIdx.x;
    if (c.q_start && c.ps_log2 > BL) {
        // two blocks to an XCD, eight workgroups apart: halves of the same lines of V may meet in its L2
        // (8000 rows, pages of 64: 24.4 -> 23.4 us)
        const int r = id % 16;
        if (id - r + 16 <= (int)gridDim.x)
            id += r % 8 * 2 + r / 8 - r;
    }
    int b = id, r0 = id, rows = 1, block = 0;
    if (c.q_start) {
        auto start = [&](int i) {
            const int64_t v = c.q_start[i];
            return (int)(v < 0 ? 0 : v < c.n_rows ? v : c.n_rows);
        };
        b = -1;
        for (int b0 = 0; b0 < c.n_seq; b0 += 256) {       // four loads in flight
            int first[4];
#pragma unroll
            for (int x = 0; x < 4; ++x)
                first[x] = start(min(b0 + 64 * x + lane, c.n_seq));
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int i = b0 + 64 * x + lane;
                b += __popcll(__ballot(i < c.n_seq && (first[x] >> BL) + 2 * i <= id));
            }
        }
        if (b < 0)
            return;
        b = __builtin_amdgcn_readfirstlane(b);
        r0 = start(b);
        rows = start(b + 1) - r0;
        block = id - ((r0 >> BL) + 2 * b);
        if (rows <= 0 || block < 0)
            return;
    }
    // positions [lo, hi) of the sequence are new; this block is positions [t0, t0 + BLOCK)
    const int64_t hi = c.kv_len[b], first = hi - rows, lo = first > 0 ? first : 0;
    const int64_t t0 = ((lo >> BL) + block) << BL;
    if (t0 >= hi)
        return;
    const int64_t entry = t0 >> c.ps_log2;
    const int page = entry < c.max_pages ? c.table[(int64_t)b * c.max_pages + entry] : -1;
    if (page < 0 || page >= c.n_pages) {
        if (tid == 0 && h == 0)
            atomicOr(c.err, 1u);
        return;
    }
    // new positions of the block: [from, to); row of position t0 + t at src + t * stride
    const int from = (int)(lo > t0 ? lo - t0 : 0), to = (int)(hi - t0 < BLOCK ? hi - t0 : BLOCK);
    const int64_t at = (r0 + (t0 - first)) * a.stride + (int64_t)h * c.hd;
    const float *ks = a.ksrc + at, *vs = a.vsrc + at;
    const int64_t out = (int64_t)page * c.page_stride + ((int64_t)h * c.hd << c.ps_log2);
    const int slot = (int)(t0 & ((1 << c.ps_log2) - 1));
    uint16_t *kd = c.k + out + (int64_t)slot * c.hd, *vd = c.v + out + slot;

    const int kp = c.hd / 8;                               // pieces of a K row
    for (int x = from * kp + tid; x < to * kp; x += 256) {
        const int t = x / kp, p = x % kp;
        const float4 u = *reinterpret_cast<const float4 *>(ks + t * a.stride + 8 * p);
        const float4 w = *reinterpret_cast<const float4 *>(ks + t * a.stride + 8 * p + 4);
        const au4 v = {pack2<T>(u.x, u.y), pack2<T>(u.z, u.w), pack2<T>(w.x, w.y), pack2<T>(w.z, w.w)};
        *reinterpret_cast<au4 *>(kd + (int64_t)t * c.hd + 8 * p) = v;
    }
    for (int x = tid; x < c.hd * PIECES_V; x += 256) {
        const int d = x / PIECES_V, t = 8 * (x % PIECES_V);
        if (t >= to || t + 8 <= from)
            continue;
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            f[e] = vs[min(max(t + e, from), to - 1) * a.stride + d];
        const au4 v = {pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]), pack2<T>(f[4], f[5]), pack2<T>(f[6], f[7])};
        uint16_t *dst = vd + ((int64_t)d << c.ps_log2) + t;
        if (t >= from && t + 8 <= to) {
            *reinterpret_cast<au4 *>(dst) = v;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (t + e >= from && t + e < to)
                    dst[e] = (uint16_t)(v[e / 2] >> (16 * (e % 2)));
        }
    }
}

// --------------------------------------------------------------- one or a few new rows per sequence
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
constexpr int JOIN_RADIX = 8;
// 16 columns; chunks of whole 128-position units, at least two; sequences of up to four are not split,
// and those of up to 32 not into more chunks than one join takes: four sequences of 4090 positions (32 / 8
// heads of 128) took 18.2 us with sixteen chunks and a second join, 15.9 with eight; one of 4090 (12 / 2)
// 10.9 and 11.2, and one of 5100 already 11.0 and 13.0.
template <bool SIDE> using AttnPlanOf = PlanOf<16, 7, 2, 4, 32, JOIN_RADIX, false, SIDE>;
typedef AttnPlanOf<false> AttnCols;

// Partial results of a slot: the tile's O (unnormalised) [cols][hd], then (exponent, sum) [cols].
// SIDE: several tiles of a KV head read the same positions.  They come next to each other and on one XCD
// (workgroups eight apart), so that one of them finds the other's in the L2: 64 sequences of 7500 positions,
// 40 / 2 heads of 128: 140.9 us tile by tile, 107 to 111; of 64 75.0 and 58; sixteen of 8 rows x 4000, 24 / 2:
// 53.3 and 47.6.  (In the code of the others it costs 0.15 of 7 us.)
template <int T, int D, bool ROWS, bool SIDE>
__global__ __launch_bounds__(256, D <= 128 ? 2 : 1) void k_attn(AttnArgs a)
{
    constexpr int KB = D / 32, DT = D / 16, NP = PIECES<T>;
    __shared__ __attribute__((aligned(16))) float s_o[4][16][D];
    __shared__ float s_m[4][16], s_l[4][16], s_mo[16], s_lo[16];
    __shared__ int s_last;
    // queries of the wide heads: every wave multiplies by the same ones, and in registers they would
    // leave none for the loads ahead
    constexpr bool Q_LDS = D > 128;
    __shared__ __attribute__((aligned(16))) au4 s_q[Q_LDS ? PIECES<T> * (D / 32) * 64 : 1];
    const KvArgs &c = a.c;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int i = lane & 15, g = lane >> 4;
    AttnPlan p;
    int id = blockIdx.x;
    if constexpr (SIDE) {
        const int run = 8 * a.side, r = id % run;
        if (id - r + run <= (int)gridDim.x)
            id += r % 8 * a.side + r / 8 - r;
    }
    if (!attn_plan<AttnPlanOf<SIDE>, ROWS>(c, a.group, attn_slots(D), id, p,
                                   reinterpret_cast<AttnSeq *>(&s_o[0][0][0])))
        return;
    const int b = p.b, chunk = p.chunk, n_chunk = p.n_chunk, len = p.len;
    const int tiles = (p.rows * a.group + 15) / 16, hkv = p.pair / tiles, rho0 = p.pair % tiles * 16;
    const int cols = min(16, p.rows * a.group - rho0);
    // offset of column col in o, and of its row and head in q
    auto head_of = [&](int col) { return hkv * a.group + (ROWS ? (rho0 + col) % a.group : rho0 + col); };
    auto row_of = [&](int col) { return p.row0 + (ROWS ? (rho0 + col) / a.group : 0); };

    // this chunk's 32-position steps, dealt to the waves in turn
    const int units = AttnCols::units(len);
    const int per = units / n_chunk, more = units % n_chunk;
    const int unit0 = chunk * per + min(chunk, more);
    const int t_begin = unit0 << AttnCols::UNIT_LOG2;
    const int t_end = min(len, (unit0 + per + (chunk < more ? 1 : 0)) << AttnCols::UNIT_LOG2);
    // positions this lane's column sees, [0, see), and those that all columns see (columns without a
    // row see what the last one does and are not stored)
    int see = t_end, see_all = t_end;
    if constexpr (ROWS) {
        const int pos0 = max(c.kv_len[b], -(1 << 30)) - p.rows;
        see = min(t_end, pos0 + (rho0 + min(i, cols - 1)) / a.group + 1);
        see_all = min(t_end, pos0 + rho0 / a.group + 1);
    }
    const int n_steps = t_end > t_begin + 32 * wave ? (t_end - t_begin - 32 * wave + 127) / 128 : 0;

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
                    s_q[(x * KB + k) * 64 + lane] = out[x];
        }
    }
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
                return s_q[(y * KB + k) * 64 + lane];
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
            uint16_t *sv = reinterpret_cast<uint16_t *>(&s_o[wave][0][0]);      // [D][32]
            if (any_bad != 0 || t + 32 > see_all) {
                if (any_bad && lane == 0)
                    atomicOr(c.err, 1u);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    sc[e] = x.bad || t + 8 * g + e >= see ? -INFINITY : sc[e];
                // what a masked position holds must not reach the product: 0 x NaN is NaN
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const int tw = t + 8 * g + 2 * w;
                    const uint32_t keep = x.bad || tw >= t_end ? 0u : tw + 1 >= t_end ? 0xFFFFu : ~0u;
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
        s_m[wave][i] = -shift;
        s_l[wave][i] = l;
    }
#pragma unroll
    for (int d = 0; d < DT; ++d)
        *reinterpret_cast<af4 *>(&s_o[wave][i][16 * d + 4 * g]) = o[d];
    __syncthreads();
    const int width = ROWS ? 16 : min(16, a.group), items = cols * (D / 4);
    const uint32_t stride = (uint32_t)attn_part_floats(width, D);
    const __amdgpu_buffer_rsrc_t part = __builtin_amdgcn_make_buffer_rsrc(
        a.part + (int64_t)p.slot0 * stride, 0, n_chunk * stride * 4, 0x00020000);
    // four channels of a column to o
    auto store = [&](int e, af4 sum, float ls) {
        const int col = e / (D / 4), d4 = e % (D / 4);
        *reinterpret_cast<af4 *>(a.o + ((int64_t)row_of(col) * a.nq + head_of(col)) * D + 4 * d4) =
            sum * inverse_sum(ls);
    };
    auto sums_at = [&](int at, int col) { return at * stride + width * D + 2 * col; };
    auto part_at = [&](int at, int e) { return at * stride + 4 * e; };

    for (int e = threadIdx.x; e < items; e += 256) {
        const int col = e / (D / 4), d4 = e % (D / 4);
        const float mm = fmaxf(fmaxf(s_m[0][col], s_m[1][col]), fmaxf(s_m[2][col], s_m[3][col]));
        af4 sum = {0.f, 0.f, 0.f, 0.f};
        float ls = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float f = join_weight(s_m[w][col], mm);
            sum += *reinterpret_cast<const af4 *>(&s_o[w][col][4 * d4]) * f;
            ls += s_l[w][col] * f;
        }
        if (n_chunk == 1) {
            store(e, sum, ls);
        } else {
            put4(part, part_at(chunk, e), sum);
            if (d4 == 0)
                put2(part, sums_at(chunk, col), mm, ls);
        }
    }
    // nodes of 1, 8, 64, ... chunks; a node's result lies in the slot of its first chunk.  The group
    // that starts at chunk g0 of level L arrives at the pair's counter g0 + L: all of a level's g0
    // are multiples of JOIN_RADIX, so no two share one
    for (int node = 1, level = 0; node < n_chunk; node *= JOIN_RADIX, ++level) {
        const int g0 = chunk / (node * JOIN_RADIX) * (node * JOIN_RADIX);
        const int members = min(JOIN_RADIX, (n_chunk - g0 + node - 1) / node);
        if (members == 1)
            continue;                                     // already in its place
        if (!last_to_arrive(a.count + p.slot0 + g0 + level, members, &s_last))
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
                store(e, sum, ls);
            } else {
                // the exponent and sum replace what other threads of the column may still have to read
                put4(part, part_at(g0, e), sum);
                if (d4 == 0) {
                    s_mo[col] = mm;
                    s_lo[col] = ls;
                }
            }
        }
        if (!top) {
            __syncthreads();
            if ((int)threadIdx.x < cols)
                put2(part, sums_at(g0, threadIdx.x), s_mo[threadIdx.x], s_lo[threadIdx.x]);
        }
    }
}

int launch_kv_append(int kv_type, const AppendArgs &a, void *stream)
{
    hipStream_t s = static_cast<hipStream_t>(stream);
    const int bl = a.c.ps_log2 < 5 ? 4 : 5;
    const int64_t blocks = a.c.q_start ? (a.c.n_rows >> bl) + 2 * (int64_t)a.c.n_seq : a.c.n_seq;
    auto k = kv_type == KV_F16 ? (bl == 4 ? k_kv_append<KV_F16, 4> : k_kv_append<KV_F16, 5>)
                               : (bl == 4 ? k_kv_append<KV_BF16, 4> : k_kv_append<KV_BF16, 5>);
    hipLaunchKernelGGL(k, dim3((unsigned)blocks, (unsigned)a.c.nkv), dim3(256), 0, s, a);
    return (int)hipGetLastError();
}

template <bool ROWS>
static int launch_k_attn(int kv_type, const AttnArgs &a, int64_t pairs, void *stream)
{
    const int slots = attn_slots(a.c.hd);
    void (*k)(AttnArgs) = nullptr;
#define QG_ATTN_D(DD)                                                                                       \
    k = kv_type == KV_F16 ? a.side > 1 ? k_attn<KV_F16, DD, ROWS, true> : k_attn<KV_F16, DD, ROWS, false>   \
                          : a.side > 1 ? k_attn<KV_BF16, DD, ROWS, true> : k_attn<KV_BF16, DD, ROWS, false>
    switch (a.c.hd) {
    case 64: QG_ATTN_D(64); break;
    case 96: QG_ATTN_D(96); break;
    case 128: QG_ATTN_D(128); break;
    case 192: QG_ATTN_D(192); break;
    default: QG_ATTN_D(256); break;
    }
#undef QG_ATTN_D
    // as many pairs as slots: those that are much longer than the rest are split all the same
    const int64_t table = (int64_t)a.c.max_pages << a.c.ps_log2;
    const int64_t grid = pairs < slots ? slots : table > AttnCols::SOLO << AttnCols::UNIT_LOG2 ? pairs + slots : pairs;
    hipLaunchKernelGGL(k, dim3((unsigned)grid), dim3(256), 0,
                       static_cast<hipStream_t>(stream), a);
    return (int)hipGetLastError();
}

int launch_attn(int kv_type, const AttnArgs &a, void *stream)
{
    AttnArgs b = a;
    b.side = (a.group + 15) / 16;
    return launch_k_attn<false>(kv_type, b, (int64_t)a.c.n_seq * a.c.nkv * b.side, stream);
}

int launch_attn_rows(int kv_type, const AttnArgs &a, void *stream)
{
    AttnArgs b = a;
    b.side = (int)((a.c.n_rows * a.group + 16 * a.c.n_seq - 1) / (16 * a.c.n_seq));   // on average
    return launch_k_attn<true>(kv_type, b, a.c.nkv * (a.c.n_rows * a.group / 16 + a.c.n_seq), stream);
}

}  // namespace qg
