// attn_prompt_kernels.hip -- causal attention of packed sequences of new rows over the paged cache.
//
// A tile is 128 rows of one sequence and one KV head, row rho = token * group + head: the query
// heads that share a KV head lie side by side, so a tile of any group spans few tokens (little of
// the diagonal is computed in vain) and every K and V element read serves all of them.  Four waves
// take 32 rows each against steps of 64 positions held in LDS.  As in the one-token kernel the
// positions are the rows of both products, S^T = K Q^T and O^T = V^T P^T (v_mfma_f32_32x32x16): a
// lane's 32 scores of a step belong to one row of the tile (column l % 32), so exponent, sum and
// factors are per-lane scalars, and they are the probabilities that the lane supplies to the second
// product (score row i of a 32-position tile is position 16 (i / 16) + 8 (i / 4 % 2) +
// 4 (i / 8 % 2) + i % 4, which makes a lane's eight values consecutive positions).
//
// K and V go from the pages to LDS without registers (global_load_lds, 16 bytes a lane), one step
// ahead, two buffers, one barrier a step.  Wave w copies the step's 16-position block w, which lies
// in one page, so page numbers and bases are scalars.  K: [position][channel], V: [block][channel]
// [16 positions].  The copies land in lane order, so the 16-byte pieces of a K row (of a V channel's
// two) are permuted at the source instead, piece ^ key of the row: a 16-byte LDS read serves 16 lanes
// (0-3, 12-15, 20-23, 24-27 and so on) from 64 banks at a time, and with these keys their 16 rows lie in
// different banks: SQ_LDS_BANK_CONFLICT 0, against four cycles a read with keys made for eight lanes
// in a row.
//
// Bound by the matrix cores: 8192 rows (32 / 8 heads of 128, f16) take 898 to 985 us from box to box, 1.22
// to 1.12 PFLOP/s with each product's two pieces counted, what a large f16 product reaches on the card; 4500
// rows of nine prompts (24 / 8 of 64, bf16, three pieces) 36 us.
#include <hip/hip_runtime.h>

#include "attn_common.h"

namespace qg {

constexpr int PT_ROWS = 128;      // rows of a tile
constexpr int PT_STEP = 64;       // positions of a step

// Global -> LDS copy of 16 bytes per lane, from base + off, to lds_dst + 16 lane.  Written as asm so
// that the compiler does not wait for it at the next LDS read: the kernel waits with vmcnt itself,
// once a step.
__device__ __forceinline__ void pt_copy16(const uint16_t *base, uint32_t off, uint32_t lds_dst)
{
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" : : "v"(off), "s"(base), "{m0}"(lds_dst) : "memory");
}
__device__ __forceinline__ void pt_wait_all()
{
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}
__device__ __forceinline__ void pt_barrier()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// 128 columns; chunks of whole steps, at least eight.  A partial result is 66 KB (heads of 128), written
// once and read once, so that up to sixteen steps are not split (one sequence of 1024 rows, 32 / 8
// heads: 39 us, in halves 59; sixteen of 32 rows behind 4000 positions: 122 us unsplit, 56).  With as many
// tiles as slots, those behind contexts longer than a slot's share are split (512 rows behind 29500
// positions beside five prompts of 307, 32 / 8 heads of 128: 842 us unsplit, 469).
typedef PlanOf<PT_ROWS, 6, 8, 16, 0, 1, true, false> PromptCols;

// A split tile, for its join.
struct PromptSplit {
    int slot0, n_chunk, row0, rows, rho0, hkv, pad[2];
};

__host__ __device__ constexpr int64_t prompt_part_floats(int hd) { return (int64_t)PT_ROWS * (hd + 2); }

// FEW: there are at least as many tiles as slots, and only those behind much longer contexts than the rest
// are split and joined in this launch (in a kernel of its own: the code of that join costs nine prompts
// without a split 36.3 -> 38.2 us).  Else, with slots, all are split and a second launch joins.
template <int T, int D, bool FEW>
__global__ __launch_bounds__(256, D <= 128 ? 2 : 1) void k_attn_prompt(AttnArgs a, int slots)
{
    constexpr int NP = PIECES<T>, KB = D / 16, DT = D / 32;
    constexpr int PR = D / 8;                          // 16-byte pieces of a K row
    // 32-position tiles of scores held at a time: three query pieces leave registers for one
    constexpr int NT = NP * D > 384 ? 1 : 2;
    // pieces that the key permutes, in pairs (heads of 256 have no registers for eight offsets)
    constexpr int KO = D == 96 ? 2 : D == 128 ? 8 : 4;
    constexpr int HALF = PT_STEP * D * 2;              // bytes of a K (or V) buffer
    constexpr int PASS = HALF / 4096;                  // copies of a wave for either
    __shared__ __attribute__((aligned(1024))) uint8_t lds[4 * HALF];   // K0 V0 K1 V1
    __shared__ int s_odd[4], s_last;
    const KvArgs &c = a.c;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 31, hf = lane >> 5;
    AttnPlan w;
    const bool work = attn_plan<PromptCols, true>(c, a.group, slots, blockIdx.x, w,
                                                  reinterpret_cast<AttnSeq *>(lds), !FEW);
    if (!FEW && blockIdx.x == 0 && tid == 0 && slots)
        *a.pairs = w.all ? w.pairs : 0;
    if (!work)
        return;
    // pairs of a sequence: tile by tile, heads side by side (the workgroups of one XCD share heads)
    struct {
        int row0, rows, rho0, pos0, hi;      // positions the tile reads: [0, hi)
    } p;
    const int hkv = w.pair % c.nkv;
    p.row0 = w.row0;
    p.rows = w.rows;
    p.rho0 = w.pair / c.nkv * PT_ROWS;
    p.pos0 = max(c.kv_len[w.b], -(1 << 30)) - p.rows;      // position of the first new row
    p.hi = max(0, min(w.len, p.pos0 + min((p.rho0 + PT_ROWS - 1) / a.group, p.rows - 1) + 1));
    // this chunk's steps, as far as the tile reads
    const int units = PromptCols::units(w.len), per = units / w.n_chunk, more = units % w.n_chunk;
    const int s0 = w.chunk * per + min(w.chunk, more);
    const int s1 = min(s0 + per + (w.chunk < more ? 1 : 0), PromptCols::units(p.hi));
    if (w.all && w.n_chunk > 1 && w.chunk == 0 && tid == 0)
        a.splits[w.first_pair + w.pair] = PromptSplit{w.slot0, w.n_chunk, p.row0, p.rows, p.rho0, hkv, {0, 0}};
    if (w.all && w.n_chunk == 1 && tid == 0)
        a.splits[w.first_pair + w.pair].n_chunk = 1;

    // this lane's row
    const int rho = p.rho0 + 32 * wave + col;
    const int tok = rho / a.group, head = hkv * a.group + rho % a.group;
    const bool live = tok < p.rows;
    // the wave's largest position (rows rise with the column); rows past the sequence compute along
    // with the last one and are not stored
    const int wave_tok0 = (p.rho0 + 32 * wave) / a.group;
    const int wave_tok1 = min((p.rho0 + 32 * wave + 31) / a.group, p.rows - 1);
    const int wave_max = wave_tok0 < p.rows ? p.pos0 + wave_tok1 : -1;
    const int pos = live ? p.pos0 + tok : wave_max;    // the row sees positions 0..pos

    au4 qf[NP][KB];
    float unscale;
    {
        const float *qr = a.q + (int64_t)(p.row0 + (live ? tok : 0)) * a.q_stride + (int64_t)head * D;
        float v[KB][8], amax = 0.f;
#pragma unroll
        for (int k = 0; k < KB; ++k) {
            const float4 x = *reinterpret_cast<const float4 *>(qr + 16 * k + 8 * hf);
            const float4 y = *reinterpret_cast<const float4 *>(qr + 16 * k + 8 * hf + 4);
            const float w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[k][e] = live ? w[e] : 0.f;
                amax = fmaxf(amax, fabsf(v[k][e]));
            }
        }
        // the mantissa of the scale goes into the queries and the rest is a power of two: scores come out
        // of their product with it exact (as their maximum is), none of either sign or zero is turned,
        // and a masked -inf stays one
        int e2 = 0;
        const float f = frexpf(a.scale, &e2) * LOG2E, sc = q_scale<T>(max_x32(amax));
        unscale = fmaxf(ldexpf(1.0f / sc, e2), 0x1p-149f);
#pragma unroll
        for (int k = 0; k < KB; ++k) {
            float w[8];
            au4 out[NP];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                w[e] = v[k][e] * sc * f;
            split8<T>(w, out);
#pragma unroll
            for (int x = 0; x < NP; ++x)
                qf[x][k] = out[x];
        }
    }

    // copies: wave w's 16-position block w.  K: piece idx = 64 x + lane of the block, row idx / PR,
    // source piece (idx % PR) ^ key(row); V: channel 32 x + lane / 2, source piece lane % 2 ^ its key
    const int32_t *table = c.table + (int64_t)w.b * c.max_pages;
    const int ps_mask = (1 << c.ps_log2) - 1;
    const int last_entry = p.hi > 0 ? (p.hi - 1) >> c.ps_log2 : 0;
    const int64_t head_off = (int64_t)hkv * D << c.ps_log2;
    const uint32_t lds0 = (uint32_t)(uintptr_t)lds;
    auto key = [](int row) { return KO == 8 ? row & 15 : KO == 4 ? (row >> 1) & 7 : (row >> 2) & 3; };
    uint32_t ksrc[PASS];
#pragma unroll
    for (int x = 0; x < PASS; ++x) {
        const int idx = 64 * x + lane, row = idx / PR;
        ksrc[x] = (uint32_t)(row * D + 8 * ((idx % PR) ^ key(row))) * 2;
    }
    const uint32_t vsrc = (uint32_t)(((lane >> 1) << c.ps_log2) + 8 * ((lane & 1) ^ (lane >> 5))) * 2;
    // page number of 16-position block lane % 4 of a step
    auto ids_of = [&](int s) { return table[min((s * PT_STEP + 16 * (lane & 3)) >> c.ps_log2, last_entry)]; };
    auto issue = [&](int s, int buf, int ids) -> uint32_t {
        const bool ok = ids >= 0 && ids < c.n_pages;
        const uint32_t bad = (uint32_t)__ballot(!ok) & 15u;
        const int page = __builtin_amdgcn_readlane(ok ? ids : 0, wave);
        const int slot = (s * PT_STEP + 16 * wave) & ps_mask;
        const int64_t at = (int64_t)page * c.page_stride + head_off;
        const uint16_t *kp = c.k + at + slot * D, *vp = c.v + at + slot;
        const uint32_t dst = lds0 + (uint32_t)(buf * 2 * HALF + wave * (HALF / 4));
#pragma unroll
        for (int x = 0; x < PASS; ++x)
            pt_copy16(kp, ksrc[x], __builtin_amdgcn_readfirstlane(dst + 1024 * x));
#pragma unroll
        for (int x = 0; x < PASS; ++x)
            pt_copy16(vp + ((32 * x) << c.ps_log2), vsrc, __builtin_amdgcn_readfirstlane(dst + HALF + 1024 * x));
        return bad;
    };

    // operand reads: K row of score row col, pieces 2 k + hf; V channel col of 32, piece hf of block k
    const int krow = 16 * (col >> 4) + 8 * ((col >> 2) & 1) + 4 * ((col >> 3) & 1) + (col & 3);
    uint32_t koff[KO];
#pragma unroll
    for (int j = 0; j < KO; ++j)
        koff[j] = (uint32_t)(krow * D * 2) + (uint32_t)(((2 * j + hf) ^ key(krow)) << 4);
    const uint32_t voff = (uint32_t)(col * 32 + ((hf ^ (col >> 4)) << 4));

    af16 o[DT];
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int r = 0; r < 16; ++r)
            o[d][r] = 0.f;
    float shift = NO_SHIFT, l = 0.f;

    // raw (unscaled) scores of positions 32 NT sub .. of a step
    auto scores = [&](int buf, int sub, af16 (&sc)[NT]) {
        const uint8_t *kb = lds + buf * 2 * HALF + sub * (NT * 64 * D);
#pragma unroll
        for (int tt = 0; tt < NT; ++tt)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                sc[tt][r] = 0.f;
        // operands are read one or two channel blocks ahead of their products (the fences keep the compiler
        // from reading all of them first, for which there are no registers)
        constexpr int AHEAD = D > 192 ? 1 : 2;
        au4 kf[AHEAD + 1][NT];
        auto read = [&](int k) {
#pragma unroll
            for (int tt = 0; tt < NT; ++tt)
                kf[k % (AHEAD + 1)][tt] = *reinterpret_cast<const au4 *>(kb + koff[k % KO] + (k / KO) * (KO * 32) + tt * 64 * D);
        };
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
            read(k);
#pragma unroll
        for (int k = 0; k < KB; ++k) {
            if (k + AHEAD < KB)
                read(k + AHEAD);
#pragma unroll
            for (int y = NP - 1; y >= 0; --y)
#pragma unroll
                for (int tt = 0; tt < NT; ++tt)
                    sc[tt] = mm32<T>(kf[k % (AHEAD + 1)][tt], qf[y][k], sc[tt]);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // scores -> probabilities (2^(score + shift)), shift and sum kept up
    auto softmax = [&](af16 (&sc)[NT]) {
        float mx = sc[0][0];
#pragma unroll
        for (int r = 0; r < 16; ++r)
#pragma unroll
            for (int tt = 0; tt < NT; ++tt)
                mx = fmaxf(mx, sc[tt][r]);
        mx *= unscale;
        if (__any(mx + shift > TOP<T>)) {
            const float to = fminf(shift, shift_of<T>(max_x32(mx)));
            const float f = __builtin_amdgcn_exp2f(to - shift);
            shift = to;
            l *= f;
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    o[d][r] *= f;
        }
        float sum[NT];
#pragma unroll
        for (int r = 0; r < 16; ++r)
#pragma unroll
            for (int tt = 0; tt < NT; ++tt) {
                sc[tt][r] = __builtin_amdgcn_exp2f(fmaf(sc[tt][r], unscale, shift));
                sum[tt] = r == 0 ? sc[tt][0] : sum[tt] + sc[tt][r];
            }
        l += NT == 2 ? sum[0] + sum[NT - 1] : sum[0];
    };
    // probability operand of 16-position block k
    auto weights = [&](const af16 (&sc)[NT], int k, au4 (&pf)[NP]) {
        float pr[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            pr[e] = sc[k >> 1][8 * (k & 1) + e];
        split8<T>(pr, pf);
    };
    // O += V^T P
    auto values = [&](const af16 (&sc)[NT], int buf, int sub) {
        const uint8_t *vb = lds + buf * 2 * HALF + HALF + sub * (NT * 64 * D);
        auto read = [&](int x) {                        // operand x = DT k + d
            return *reinterpret_cast<const au4 *>(vb + voff + (x / DT) * (D * 32) + (x % DT) * 1024);
        };
        constexpr int AHEAD = D > 192 ? 2 : 3;
        au4 v[AHEAD + 1], pf[NP];
#pragma unroll
        for (int x = 0; x < AHEAD; ++x)
            v[x] = read(x);
#pragma unroll
        for (int x = 0; x < 2 * NT * DT; ++x) {
            if (x + AHEAD < 2 * NT * DT)
                v[(x + AHEAD) % (AHEAD + 1)] = read(x + AHEAD);
            if (x % DT == 0)
                weights(sc, x / DT, pf);
#pragma unroll
            for (int y = NP - 1; y >= 0; --y)
                o[x % DT] = mm32<T>(v[x % (AHEAD + 1)], pf[y], o[x % DT]);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // Edge steps hold positions that some rows of the tile do not see.  An infinity or NaN in V there
    // must reach the rows that see it and no other, but 0 x NaN is NaN: such values are added to
    // their rows one by one and then cleared in LDS.
    constexpr int SUB = NT * 64 * D;                    // bytes of V that belong to NT tiles
    auto scan = [&](int buf) {
        uint32_t nf = 0;
#pragma unroll 1
        for (int x = tid; x < HALF / 16; x += 256) {
            const au4 v = *reinterpret_cast<const au4 *>(lds + buf * 2 * HALF + HALF + 16 * x);
            nf |= nonfinite2<T>(v[0]) | nonfinite2<T>(v[1]) | nonfinite2<T>(v[2]) | nonfinite2<T>(v[3]);
        }
        s_odd[wave] = __any(nf != 0);
        __syncthreads();
        return (s_odd[0] | s_odd[1] | s_odd[2] | s_odd[3]) != 0;
    };
    auto clear = [&](int buf, int sub) {
#pragma unroll 1
        for (int x = tid; x < SUB / 16; x += 256) {
            au4 *v = reinterpret_cast<au4 *>(lds + buf * 2 * HALF + HALF + sub * SUB + 16 * x);
            au4 y = *v;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const uint32_t nf = nonfinite2<T>(y[w]);
                y[w] &= ~((nf - (nf >> 15)) | nf);
            }
            *v = y;
        }
    };
    auto add_nonfinite = [&](int see, uint32_t bad, int buf, int sub) {
        const uint8_t *vb = lds + buf * 2 * HALF + HALF;
#pragma unroll 1
        for (int t = 32 * NT * sub; t < 32 * NT * (sub + 1); ++t) {
            if (bad >> (t >> 4) & 1)
                continue;
            const uint32_t at = (t >> 4) * (D * 32) + 2 * (t & 7);
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int ch = 8 * (r >> 2) + 4 * hf + (r & 3);      // channel 32 d + ch
                    const uint16_t x = *reinterpret_cast<const uint16_t *>(
                        vb + at + d * 1024 + ch * 32 + ((((t >> 3) & 1) ^ (ch >> 4)) << 4));
                    if (t <= see && nonfinite2<T>(x))
                        o[d][r] += low_of<T>(x);
                    if (r % 8 == 7)
                        __builtin_amdgcn_sched_barrier(0);
                }
        }
    };
    // the tile's least position; a table that ends before it may end inside a step
    const int tile_min = min(p.pos0 + p.rho0 / a.group, p.hi - 1);
    auto compute = [&](int s, int buf, uint32_t bad) {
        const int t0 = s * PT_STEP;
        const bool edge = bad != 0 || t0 + PT_STEP - 1 > tile_min;
        const bool odd = edge ? scan(buf) : false;
        const bool active = t0 <= wave_max;            // else nothing of this step is seen by the wave
        const int see = min(pos, p.hi - 1) - t0;
#pragma unroll
        for (int sub = 0; sub < 2 / NT; ++sub) {
            af16 sc[NT];
            if (active) {
                scores(buf, sub, sc);
                // value r of tile tt is position t0 + 32 (NT sub + tt) + 16 (r / 8) + 8 hf + r % 8
                if (edge)
#pragma unroll
                    for (int tt = 0; tt < NT; ++tt)
#pragma unroll
                        for (int r = 0; r < 16; ++r) {
                            const int blk = 2 * (NT * sub + tt) + (r >> 3);
                            if (16 * blk + (r & 7) > see - 8 * hf || (bad >> blk & 1))
                                sc[tt][r] = -INFINITY;
                        }
                softmax(sc);
            }
            if (odd) {
                if (active)
                    add_nonfinite(see, bad, buf, sub);
                __syncthreads();
                clear(buf, sub);
                __syncthreads();
            }
            if (active)
                values(sc, buf, sub);
        }
    };

    if (s1 > s0) {
        uint32_t bad_next = issue(s0, 0, ids_of(s0)), seen_bad = 0;
        int ids = ids_of(s0 + 1);
        for (int s = s0; s < s1; ++s) {
            const int buf = (s - s0) & 1;
            const uint32_t bad = bad_next;
            seen_bad |= bad;
            // this thread's copies of step s have landed; after the barrier everyone's have, and
            // everyone is done with step s - 1, whose buffer the next copies overwrite
            pt_wait_all();
            pt_barrier();
            if (s + 1 < s1) {
                bad_next = issue(s + 1, buf ^ 1, ids);
                ids = ids_of(s + 2);
            }
            compute(s, buf, bad);
        }
        if (seen_bad && tid == 0)
            atomicOr(c.err, 1u);
    }

    // O^T: lane's row, channels 32 d + 8 (r / 4) + 4 hf + r % 4
    l = sum_x32(l);
    if (!FEW && w.n_chunk > 1) {
        float *part = a.part + (int64_t)(w.slot0 + w.chunk) * prompt_part_floats(D);
        float *row = part + (32 * wave + col) * D + 4 * hf;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                *reinterpret_cast<af4 *>(row + 32 * d + 8 * r) =
                    af4{o[d][4 * r], o[d][4 * r + 1], o[d][4 * r + 2], o[d][4 * r + 3]};
        if (hf == 0) {
            float *ml = part + PT_ROWS * D + 2 * (32 * wave + col);
            ml[0] = -shift;
            ml[1] = l;
        }
        return;
    }
    if (FEW && w.n_chunk > 1) {
        // one of a few split tiles among many whole ones: the last of its workgroups to finish adds the
        // parts, in the order of the chunks
        const uint32_t stride = (uint32_t)prompt_part_floats(D);
        const __amdgpu_buffer_rsrc_t part = __builtin_amdgcn_make_buffer_rsrc(
            a.part + (int64_t)w.slot0 * stride, 0, w.n_chunk * stride * 4, 0x00020000);
        const uint32_t row = (32 * wave + col) * D + 4 * hf, ml = PT_ROWS * D + 2 * (32 * wave + col);
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                put4(part, w.chunk * stride + row + 32 * d + 8 * r,
                     af4{o[d][4 * r], o[d][4 * r + 1], o[d][4 * r + 2], o[d][4 * r + 3]});
        if (hf == 0)
            put2(part, w.chunk * stride + ml, -shift, l);
        if (!last_to_arrive(a.count + w.slot0, w.n_chunk, &s_last))
            return;
        float m = -INFINITY;
        for (int k = 0; k < w.n_chunk; ++k) {
            float mk, lk;
            get2(part, k * stride + ml, mk, lk);
            m = fmaxf(m, mk);
        }
        l = 0.f;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                o[d][r] = 0.f;
#pragma unroll 1
        for (int k = 0; k < w.n_chunk; ++k) {
            float mk, lk;
            get2(part, k * stride + ml, mk, lk);
            const float f = join_weight(mk, m);
            af4 x[DT][4];
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    x[d][r] = get4(part, k * stride + row + 32 * d + 8 * r);
            l += lk * f;
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    o[d][r] += x[d][r / 4][r % 4] * f;
        }
    }
    if (live) {
        const float inv = inverse_sum(l);
        float *row = a.o + ((int64_t)(p.row0 + tok) * a.nq + head) * D + 4 * hf;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                *reinterpret_cast<af4 *>(row + 32 * d + 8 * r) =
                    af4{o[d][4 * r] * inv, o[d][4 * r + 1] * inv, o[d][4 * r + 2] * inv, o[d][4 * r + 3] * inv};
    }
}

// Rows of a split tile from its partial results.  A workgroup takes four rows of a tile and KV head at a
// time; a thread four channels of a row and every `parts`-th split, in order, then the parts are added
// in order.
__global__ __launch_bounds__(256) void k_attn_prompt_join(AttnArgs a)
{
    __shared__ __attribute__((aligned(16))) af4 s_sum[256];
    __shared__ float s_m[256], s_l[256];
    if ((int)blockIdx.x >= *a.pairs)
        return;
    const PromptSplit p = a.splits[blockIdx.x];
    const int splits = p.n_chunk;
    if (splits <= 1)
        return;
    const int D = a.c.hd, lanes = D / 4, items = 4 * lanes, parts = 256 / items;
    const int tid = threadIdx.x, e = tid % items, k0 = tid / items, row = e / lanes, d4 = e % lanes;
    const int64_t stride = prompt_part_floats(D);
    for (int r0 = 4 * blockIdx.y; r0 < PT_ROWS && (p.rho0 + r0) / a.group < p.rows; r0 += 4 * gridDim.y) {
        const float *part = a.part + p.slot0 * stride, *from = part + (r0 + row) * D + 4 * d4;
        const float *ml = part + PT_ROWS * D + 2 * (r0 + row);
        float m = -INFINITY, l = 0.f;
        af4 sum = {0.f, 0.f, 0.f, 0.f};
        for (int kb = k0; k0 < parts && kb < splits; kb += 8 * parts) {
            af4 v[8];
            float2 w[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) {                      // all loads in flight at once
                const int64_t at = min(kb + x * parts, splits - 1) * stride;
                w[x] = *reinterpret_cast<const float2 *>(ml + at);
                v[x] = *reinterpret_cast<const af4 *>(from + at);
            }
            float mb = m;
#pragma unroll
            for (int x = 0; x < 8; ++x)
                mb = fmaxf(mb, w[x].x);
            const float f0 = join_weight(m, mb);
            sum *= f0;
            l *= f0;
            m = mb;
#pragma unroll
            for (int x = 0; x < 8; ++x)
                if (kb + x * parts < splits) {
                    const float f = join_weight(w[x].x, m);
                    sum += v[x] * f;
                    l += w[x].y * f;
                }
        }
        if (parts > 1) {
            s_sum[tid] = sum;
            s_m[tid] = m;
            s_l[tid] = l;
            __syncthreads();
            if (k0 == 0) {
                float all = m;
                for (int x = 1; x < parts; ++x)
                    all = fmaxf(all, s_m[e + x * items]);
                const float f0 = join_weight(m, all);
                sum *= f0;
                l *= f0;
                for (int x = 1; x < parts; ++x) {
                    const float f = join_weight(s_m[e + x * items], all);
                    sum += s_sum[e + x * items] * f;
                    l += s_l[e + x * items] * f;
                }
            }
            __syncthreads();
        }
        const int rho = p.rho0 + r0 + row, tok = rho / a.group;
        if (k0 == 0 && tok < p.rows)
            *reinterpret_cast<af4 *>(a.o + ((int64_t)(p.row0 + tok) * a.nq + p.hkv * a.group + rho % a.group) * D +
                                     4 * d4) = sum * inverse_sum(l);
    }
}

// Pairs (tiles times KV heads) of a call at most; whether any may be split (the table holds more positions
// than a chunk alone takes); and whether that is for having fewer than slots, so that a second launch joins
// them, or for being longer than others (the tiles of one sequence are alike).
PromptPlan plan_prompt(int64_t n_rows, int n_seq, int nkv, int group, int hd, int64_t positions)
{
    PromptPlan p;
    p.pairs = nkv * (n_rows * group / PT_ROWS + n_seq);
    const bool may = positions > (PromptCols::SOLO << PromptCols::UNIT_LOG2);
    // (a sequence's last tile is half full on average)
    p.second = may && nkv * (n_rows * group / PT_ROWS + n_seq / 2) < prompt_slots(hd) && p.pairs <= PROMPT_SPLITS;
    p.slots = p.second || (may && n_seq > 1) ? prompt_slots(hd) : 0;
    p.grid = !p.second ? p.pairs + p.slots : p.pairs > p.slots ? p.pairs : p.slots;
    return p;
}

// Few columns (rows times query heads of a KV head): the one-token kernel takes 16 at a time, with the
// positions spread over all waves, where this one's 128-row tiles would mostly be empty or too few.  It
// reads the cache once per 16 columns, so it takes the call when all its workgroups are resident at once, the
// columns of a sequence are at most 384 on average or the table is short, and the whole work is bounded
// however the rows are dealt to the sequences, which only the device knows: every column times every position
// of the table stays under 2^31 channels (of longer tables 16384 positions count: a table is sized for the
// longest cache, and the 16-column tiles are done 20 us earlier where it is not full).
// 128-row tiles -> 16 columns, us: 16 sequences x 4 rows x 4000 positions, 32 / 8 heads of 128, 64.7 -> 38.9;
// one of 32 rows x 20000, 12 / 2 heads, 36.3 -> 34.1; of 128 rows 57.9 -> 84.1; three of 31 rows alone
// 9.6 -> 6.8; one of 128 rows alone, 32 / 8 heads, 11.4 -> 8.4; 16 of 32 rows alone, twice the resident
// workgroups, 11.0 -> 19.9; four of 32 rows x 2000, 12 / 2, 29.9 -> 21.8; 177 rows behind 30000 positions
// among 15 single tokens, 24 / 2 heads (156 columns on average), 139 -> 528.  Over 1119 mixes of rows and
// caches, heads of 64 to 256, the choice costs 2.7 % against the faster one each; without the bound on the
// work 11.8 %, and 280 % at worst.  64 sequences of 4 rows x 4000 positions would gain as well (189.7 ->
// 181.9, at 8 rows 192 -> 285), but as many rows may be one prompt among single tokens.
bool prompt_in_16s(int64_t n_rows, int n_seq, int nq, int nkv, int hd, int64_t positions)
{
    const int64_t columns = n_rows * (nq / nkv);
    return nkv * (columns / 16 + n_seq) <= attn_slots(hd) && (columns <= 384 * (int64_t)n_seq || positions <= 1024) &&
           columns * nkv * hd * (positions < 16384 ? positions : 16384) <= (int64_t)1 << 31;
}

int launch_attn_prompt(int kv_type, const AttnArgs &a, void *stream)
{
    const int64_t table = (int64_t)a.c.max_pages << a.c.ps_log2;
    if (prompt_in_16s(a.c.n_rows, a.c.n_seq, a.nq, a.c.nkv, a.c.hd, table))
        return launch_attn_rows(kv_type, a, stream);
    hipStream_t s = static_cast<hipStream_t>(stream);
    const PromptPlan p = plan_prompt(a.c.n_rows, a.c.n_seq, a.c.nkv, a.group, a.c.hd, table);
    const bool few = p.slots && !p.second;
    void (*k)(AttnArgs, int) = nullptr;
#define QG_PROMPT_D(DD)                                                                                  \
    k = kv_type == KV_F16 ? few ? k_attn_prompt<KV_F16, DD, true> : k_attn_prompt<KV_F16, DD, false>     \
                          : few ? k_attn_prompt<KV_BF16, DD, true> : k_attn_prompt<KV_BF16, DD, false>
    switch (a.c.hd) {
    case 64: QG_PROMPT_D(64); break;
    case 96: QG_PROMPT_D(96); break;
    case 128: QG_PROMPT_D(128); break;
    case 192: QG_PROMPT_D(192); break;
    default: QG_PROMPT_D(256); break;
    }
#undef QG_PROMPT_D
    hipLaunchKernelGGL(k, dim3((unsigned)p.grid), dim3(256), 0, s, a, p.slots);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !p.second)
        return (int)e;
    // the fewer tiles, the more workgroups share one, about 4096 in all (sixteen sequences of 32 rows
    // behind 4000 positions: 56.3 us, with 2048 61.4; 8192 that find nothing to join cost 1 us more)
    const int64_t share = 4096 / p.pairs;
    const unsigned y = (unsigned)(share > PT_ROWS / 4 ? PT_ROWS / 4 : share > 8 ? share : 8);
    hipLaunchKernelGGL(k_attn_prompt_join, dim3((unsigned)p.pairs, y), dim3(256), 0, s, a);
    return (int)hipGetLastError();
}

}  // namespace qg
