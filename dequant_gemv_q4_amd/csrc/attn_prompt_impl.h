// attn_prompt_impl.h -- causal attention of packed sequences of new rows over the paged cache.
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
// rows of nine prompts (24 / 8 of 64, bf16, three pieces) 36 us.  Over 8-bit pages the vector instructions (scales,
// conversions, softmax: 500 a step of 64 positions with its 64 products, heads of 128) nearly reach the products' time:
// I8 1020 to 1050 us for the same rows, F8 1000 to 1020, the nine prompts 39 us.
#pragma once

#include <float.h>

#include "attn_bytes.h"

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

// LDS of a workgroup.
template <int T, int D>
struct PromptLds {
    static constexpr int HALF = PT_STEP * D * 2;
    __attribute__((aligned(1024))) uint8_t kv[4 * HALF];               // K0 V0 K1 V1
    float scale[kv_bytes(T) ? 2 : 1][2][PT_STEP];                      // 8-bit: of K and V
    int odd[4], most[4], last;
};

// FEW: there are at least as many tiles as slots, and only those behind much longer contexts than the rest
// are split and joined in this launch (in a kernel of its own: the code of that join costs nine prompts
// without a split 36.3 -> 38.2 us).  Else, with slots, all are split and a second launch joins.
// SHARED: the rows are the sequences of a group, and see its shared positions (PREFIX); what each sees behind
// them is in o and stats.  JOINED: that is added here, to tiles that are not split or by the last of a tile's
// workgroups; PARTED: all tiles leave parts (beside the workgroups that fill o and stats), and the next launch
// joins.
enum PromptForm { CAUSAL, JOINED, PARTED };
template <int T, int D, bool FEW, int SHARED>
__device__ __forceinline__ void prompt_body(const AttnArgs &a, int slots, int id, PromptLds<T, D> &sh)
{
    constexpr bool BYTES = kv_bytes(T);
    constexpr int F = BYTES ? KV_F16 : T;              // operands of the products
    constexpr int NP = PIECES<F>, KB = D / 16, DT = D / 32;
    constexpr int PR = D / 8;                          // 16-byte pieces of a K row
    // 32-position tiles of scores held at a time: three query pieces leave registers for one
    constexpr int NT = NP * D > 384 ? 1 : 2;
    // pieces that the key permutes, in pairs (heads of 256 have no registers for eight offsets)
    constexpr int KO = D == 96 ? 2 : D == 128 ? 8 : 4;
    constexpr int HALF = PromptLds<T, D>::HALF;        // bytes of a K (or V) buffer
    constexpr int PASS = HALF / 4096;                  // copies of a wave for either
    uint8_t *const lds = sh.kv;
    const KvArgs &c = a.c;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 31, hf = lane >> 5;
    AttnPlan w;
    const bool work = attn_plan<PromptCols, SHARED ? PREFIX : MANY>(a, slots, id, w,
                                                                    reinterpret_cast<AttnSeq *>(lds), !FEW);
    if (!FEW && id == 0 && tid == 0 && slots)
        *a.pairs = w.all ? w.pairs : 0;
    if (!work || (SHARED == PARTED && (!w.all || w.slot0 + w.n_chunk > slots)))
        return;
    // pairs of a sequence: tile by tile, heads side by side (the workgroups of one XCD share heads)
    struct {
        int row0, rows, rho0, pos0, hi;      // positions the tile reads: [0, hi)
    } p;
    const int hkv = w.pair % c.nkv;
    p.row0 = w.row0;
    p.rows = w.rows;
    p.rho0 = w.pair / c.nkv * PT_ROWS;
    p.pos0 = SHARED ? 0 : max(c.kv_len[w.b], -(1 << 30)) - p.rows;      // position of the first new row
    p.hi = SHARED ? w.len : max(0, min(w.len, p.pos0 + min((p.rho0 + PT_ROWS - 1) / a.group, p.rows - 1) + 1));
    // this chunk's steps, as far as the tile reads
    const int units = PromptCols::units(w.len), per = units / w.n_chunk, more = units % w.n_chunk;
    const int s0 = w.chunk * per + min(w.chunk, more);
    if (w.all && (w.n_chunk > 1 || SHARED == PARTED) && w.chunk == 0 && tid == 0)
        a.splits[w.first_pair + w.pair] = PromptSplit{w.slot0, w.n_chunk, p.row0, p.rows, p.rho0, hkv, {0, 0}};
    if (w.all && w.n_chunk == 1 && SHARED != PARTED && tid == 0)
        a.splits[w.first_pair + w.pair].n_chunk = 1;

    // this lane's row
    const int rho = p.rho0 + 32 * wave + col;
    const int tok = rho / a.group, head = hkv * a.group + rho % a.group;
    const bool live = tok < p.rows;
    // the wave's largest position (rows rise with the column); rows past the sequence compute along
    // with the last one and are not stored
    const int wave_tok0 = (p.rho0 + 32 * wave) / a.group;
    const int wave_tok1 = min((p.rho0 + 32 * wave + 31) / a.group, p.rows - 1);
    int wave_max = wave_tok0 < p.rows ? p.pos0 + wave_tok1 : -1;
    int pos = live ? p.pos0 + tok : wave_max;          // the row sees positions 0..pos
    // the tile's least position; a table that ends before it may end inside a step
    int tile_min = min(p.pos0 + p.rho0 / a.group, p.hi - 1);
    if constexpr (SHARED) {
        // (positions of a table are below 2^24, whole numbers in f32)
        pos = live ? prefix_seen(a, p.row0 + tok, w.len) - 1 : -1;
        wave_max = __builtin_amdgcn_readfirstlane((int)max_x16(max_of_16((float)pos)));
        const int least = -(int)max_x16(max_of_16(live ? -(float)pos : -(float)p.hi));
        sh.odd[wave] = __builtin_amdgcn_readfirstlane(least);
        sh.most[wave] = wave_max;
        __syncthreads();
        // what none of the tile's rows sees is not read
        const int most = max(max(sh.most[0], sh.most[1]), max(sh.most[2], sh.most[3]));
        p.hi = min(p.hi, __builtin_amdgcn_readfirstlane(most) + 1);
        tile_min = min(min(sh.odd[0], sh.odd[1]), min(sh.odd[2], sh.odd[3]));
        tile_min = min(__builtin_amdgcn_readfirstlane(tile_min), p.hi - 1);
        __syncthreads();
    }
    const int s1 = min(s0 + per + (w.chunk < more ? 1 : 0), PromptCols::units(p.hi));

    au4 qf[NP][KB];
    float unscale;
    float k_room = 1.0f;                               // (uniform)
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
        const float f = frexpf(a.scale, &e2) * LOG2E, sc = q_scale<F>(max_x32(amax));
        unscale = fmaxf(ldexpf(1.0f / sc, e2), 0x1p-149f);
        // 8-bit: a product times K's scale must not leave f32 where unscale brings the score back, and with K_ROOM of
        // the scale it does not.  What that takes from scales below 2^-94 is nothing to a score (2^-26 of its
        // exponent), unless queries are so near f32's end that it could be: then scales stay as they are.  (8192
        // rows, 32 / 8 heads of 128, I8, 1016 -> 1021 us; a vote on the scales of each step instead 1027.)
        if constexpr (BYTES) {
            k_room = scalar(__any(unscale > 0x1p60f) ? 1.0f : K_ROOM);
            unscale *= 1.0f / k_room;
        }
#pragma unroll
        for (int k = 0; k < KB; ++k) {
            float w[8];
            au4 out[NP];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                w[e] = v[k][e] * sc * f;
            split8<F>(w, out);
#pragma unroll
            for (int x = 0; x < NP; ++x)
                qf[x][k] = out[x];
        }
    }

    // copies: wave w's 16-position block w.  K: piece idx = 64 x + lane of the block, row idx / PR,
    // source piece (idx % PR) ^ key(row); V: channel 32 x + lane / 2, source piece lane % 2 ^ its key
    const int32_t *table = c.table + (int64_t)(SHARED ? p.row0 : w.b) * c.max_pages;
    const int ps_mask = (1 << c.ps_log2) - 1;
    const int last_entry = p.hi > 0 ? (p.hi - 1) >> c.ps_log2 : 0;
    const int64_t head_off = BYTES ? (int64_t)hkv * c.block : (int64_t)hkv * D << c.ps_log2;
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
    // 8-bit pages: the same block of a step goes through registers, 16 codes a lane, and to LDS as f16 where
    // the copies would have put it; lanes 0-15 carry the scales of K, lanes 16-31 those of V
    constexpr int PASS8 = (D + 63) / 64;
    struct Codes {
        au4 k[PASS8], v[PASS8];
        float d;
        uint32_t bad;
    };
    auto load8 = [&](int s, int ids, Codes &x) {
        const bool ok = ids >= 0 && ids < c.n_pages;
        x.bad = (uint32_t)__ballot(!ok) & 15u;
        const int page = __builtin_amdgcn_readlane(ok ? ids : 0, wave);
        const int slot = (s * PT_STEP + 16 * wave) & ps_mask;
        const int64_t at = (int64_t)page * c.page_stride + head_off;
        const uint8_t *kp = c.k8() + at + slot * D, *vp = c.v8() + at + slot;
        const uint8_t *dp = (lane & 16 ? c.v8() : c.k8()) + at + ((int64_t)D << c.ps_log2) + 4 * slot;
        x.d = reinterpret_cast<const float *>(dp)[lane & 15];
#pragma unroll
        for (int i = 0; i < PASS8; ++i) {
            const int idx = min(64 * i + lane, D - 1);
            x.k[i] = *reinterpret_cast<const au4 *>(kp + 16 * idx);
            x.v[i] = *reinterpret_cast<const au4 *>(vp + ((int64_t)idx << c.ps_log2));
        }
    };
    auto stage8 = [&](int s, int buf, Codes &x) {
        uint8_t *kb = lds + buf * 2 * HALF + wave * (HALF / 4), *vb = kb + HALF;
        const int left = x.bad >> wave & 1 ? 0 : p.hi - s * PT_STEP - 16 * wave;   // positions of the block
        if (left < 16) {
            // what a masked position holds must not reach the product: an e4m3 may be NaN
            if constexpr (T == KV_F8)
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const int m = left - 4 * w;
                    const uint32_t keep = m >= 4 ? ~0u : m <= 0 ? 0u : (1u << (8 * m)) - 1u;
#pragma unroll
                    for (int i = 0; i < PASS8; ++i)
                        x.v[i][w] &= keep;
                }
            x.d = (lane & 15) < left ? x.d : 0.f;
        }
        if (lane < 32)
            sh.scale[BYTES ? buf : 0][lane >> 4][16 * wave + (lane & 15)] = x.d;
        // K and V apart (I8, 8192 rows, 32 / 8 heads of 128, 1072 -> 1027 us, 4096 of 256 822 -> 749 against a loop
        // body for both, which the compiler orders worse)
#pragma unroll
        for (int n = 0; n < 2 * PASS8; ++n) {
            const int idx = 64 * (n / 2) + lane, row = idx / (D / 16), pc = 2 * (idx % (D / 16));
            if (D % 64 == 0 || idx < D) {
                au4 lo, hi;
                if (n % 2 == 0) {
                    halves_of<T>(x.k[n / 2], lo, hi);
                    *reinterpret_cast<au4 *>(kb + row * D * 2 + ((pc ^ key(row)) << 4)) = lo;
                    *reinterpret_cast<au4 *>(kb + row * D * 2 + (((pc + 1) ^ key(row)) << 4)) = hi;
                } else {
                    halves_of<T>(x.v[n / 2], lo, hi);
                    const int turn = idx >> 4 & 1;
                    *reinterpret_cast<au4 *>(vb + idx * 32 + (turn << 4)) = lo;
                    *reinterpret_cast<au4 *>(vb + idx * 32 + ((turn ^ 1) << 4)) = hi;
                }
            }
        }
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
    // 8-bit: the wave's reference of V's scales, the row's largest scale above it
    float ref = -200.0f, top = LEAST_TOP;

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
                    sc[tt] = mm32<F>(kf[k % (AHEAD + 1)][tt], qf[y][k], sc[tt]);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // 8-bit: position of lane i of each 16 in tile x of a step, so that value r of a row is lane r's
    auto scale_at = [&](int x) { return 32 * x + 16 * ((lane & 15) >> 3) + 8 * hf + (lane & 7); };
    // scores -> probabilities (2^(score + shift)), shift and sum kept up.  most: 8-bit, the largest exponent of V's
    // scales that a row of the wave sees
    auto softmax = [&](af16 (&sc)[NT], float most) {
        float mx = sc[0][0];
#pragma unroll
        for (int r = 0; r < 16; ++r)
#pragma unroll
            for (int tt = 0; tt < NT; ++tt)
                mx = fmaxf(mx, sc[tt][r]);
        mx *= unscale;
        const bool moved = BYTES && __builtin_amdgcn_readfirstlane(most > ref + R_SLACK);
        if (__any(moved || (BYTES ? mx + shift > TOP8 - top : mx + shift > TOP<F>))) {
            float f;
            if constexpr (BYTES) {
                const float to = moved ? scalar(most) : ref;
                const Rescaled x = rescaled(ref, to, top, shift, max_x32(mx), exponent_above(max_x32(l)));
                ref = to;
                top = x.top;
                shift = x.shift;
                l *= x.l;
                f = x.o;
            } else {
                const float to = fminf(shift, shift_of<F>(max_x32(mx)));
                f = __builtin_amdgcn_exp2f(to - shift);
                shift = to;
                l *= f;
            }
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
        split8<F>(pr, pf);
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
                o[x % DT] = mm32<F>(v[x % (AHEAD + 1)], pf[y], o[x % DT]);
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
        sh.odd[wave] = __any(nf != 0);
        __syncthreads();
        return (sh.odd[0] | sh.odd[1] | sh.odd[2] | sh.odd[3]) != 0;
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
    // between: what is done between the two products (loads of 8-bit pages there: 8192 rows, 32 / 8 heads of 128, F8
    // 1104 -> 1050 us against before both)
    auto compute = [&](int s, int buf, uint32_t bad, auto between) {
        const int t0 = s * PT_STEP;
        const bool edge = bad != 0 || t0 + PT_STEP - 1 > tile_min;
        const bool odd = !BYTES && edge ? scan(buf) : false;
        const bool active = t0 <= wave_max;            // else nothing of this step is seen by the wave
        const int see = min(pos, p.hi - 1) - t0;
        // Whether the row does not see value r of tile tt, from the last position that it sees.  8-bit: made anew in
        // each branch that asks, else the compiler makes the 32 comparisons in every step ahead of the branches; with
        // these asked less often (nine prompts, 4500 rows, 24 / 8 heads of 64, F8, 46.5 -> 43.0 us, I8, 8192 rows,
        // 32 / 8 of 128, 1084 -> 1045; f16 and bf16 the same or 1 % slower).
        auto last_seen = [&]() {
            int last = see - 8 * hf;
            if constexpr (BYTES)
                asm volatile("" : "+v"(last));
            return last;
        };
        auto hidden = [&](int last, int sub, int tt, int r) {
            const int blk = 2 * (NT * sub + tt) + (r >> 3);
            return (r & 7) > (bad >> blk & 1 ? -1 : last - 16 * blk);
        };
#pragma unroll
        for (int sub = 0; sub < 2 / NT; ++sub) {
            af16 sc[NT];
            if (active) {
                scores(buf, sub, sc);
                float dv[NT];
                if constexpr (BYTES)
#pragma unroll
                    for (int tt = 0; tt < NT; ++tt) {
                        const int at = scale_at(NT * sub + tt);
                        dv[tt] = sh.scale[buf][1][at];
                        times_lanes([&](int r) { return Ref<af16>{sc[tt], r}; }, sh.scale[buf][0][at] * k_room);
                    }
                // value r of tile tt is position t0 + 32 (NT sub + tt) + 16 (r / 8) + 8 hf + r % 8
                if (edge) {
                    const int last = last_seen();
#pragma unroll
                    for (int tt = 0; tt < NT; ++tt)
#pragma unroll
                        for (int r = 0; r < 16; ++r)
                            if (hidden(last, sub, tt, r))
                                sc[tt][r] = -INFINITY;
                }
                float most = 0.f;
                if constexpr (BYTES) {
                    float seen = dv[0];
                    if constexpr (NT == 2)
                        seen = fmaxf(seen, dv[NT - 1]);
                    seen = max_x32(max_of_16(seen));
                    most = exponent_above(seen);
                    // scales that some rows do not see matter where they pass what a row has seen
                    if (edge && __any(most > ref + top)) {
                        const int last = last_seen();
                        seen = 0.f;
#pragma unroll
                        for (int tt = 0; tt < NT; ++tt)
                            each_lane([&](int r, float d) { seen = hidden(last, sub, tt, r) ? seen : fmaxf(seen, d); },
                                      dv[tt]);
                        seen = max_x32(seen);
                        most = max_x16(max_of_16(exponent_above(seen)));
                    }
                    top = fmaxf(top, exponent_above(seen) - ref);
                }
                softmax(sc, most);
                if constexpr (BYTES)
#pragma unroll
                    for (int tt = 0; tt < NT; ++tt) {
                        dv[tt] = ldexpf(dv[tt], -(int)ref);
                        times_lanes([&](int r) { return Ref<af16>{sc[tt], r}; }, dv[tt]);
                        if (edge && __any(!(dv[tt] <= FLT_MAX))) {       // a NaN scale that this row does not see
                            const int last = last_seen();
#pragma unroll
                            for (int r = 0; r < 16; ++r)
                                sc[tt][r] = hidden(last, sub, tt, r) ? 0.f : sc[tt][r];
                        }
                    }
            }
            if (odd) {
                if (active)
                    add_nonfinite(see, bad, buf, sub);
                __syncthreads();
                clear(buf, sub);
                __syncthreads();
            }
            if (sub == 0)
                between();
            if (active)
                values(sc, buf, sub);
        }
    };

    if (BYTES && s1 > s0) {
        // a step's loads are under way while the one before is computed: all of it where there are registers for
        // that, else between its products
        constexpr bool AHEAD = D <= 96;
        Codes x;
        load8(s0, ids_of(s0), x);
        int ids = ids_of(s0 + 1);
        stage8(s0, 0, x);
        uint32_t bad = x.bad, seen_bad = 0;
        auto next = [&](int s) {
            if (s < s1) {
                load8(s, ids, x);
                ids = ids_of(s + 1);
            }
        };
        if (AHEAD)
            next(s0 + 1);
        for (int s = s0; s < s1; ++s) {
            const int buf = (s - s0) & 1;
            seen_bad |= bad;
            // step s is staged; after the barrier everyone's part is, and everyone is done with step s - 1
            __syncthreads();
            compute(s, buf, bad, [&]() {
                if (!AHEAD)
                    next(s + 1);
            });
            if (s + 1 < s1) {
                stage8(s + 1, buf ^ 1, x);
                bad = x.bad;
                if (AHEAD)
                    next(s + 2);
            }
        }
        if (seen_bad && tid == 0)
            atomicOr(c.err, 1u);
    } else if (s1 > s0) {
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
            compute(s, buf, bad, []() {});
        }
        if (seen_bad && tid == 0)
            atomicOr(c.err, 1u);
    }

    // O^T: lane's row, channels 32 d + 8 (r / 4) + 4 hf + r % 4
    l = sum_x32(l);
    if constexpr (BYTES) {                             // parts are means
        const float inv = inverse_sum(l);
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                o[d][r] = ldexpf(o[d][r] * inv, (int)ref);
    }
    if (!FEW && (w.n_chunk > 1 || SHARED == PARTED)) {
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
        if (!last_to_arrive(a.count + w.slot0, w.n_chunk, &sh.last))
            return;
        float m = -INFINITY;
        for (int k = 0; k < w.n_chunk; ++k) {
            float mk, lk;
            get2(part, k * stride + ml, mk, lk);
            m = fmaxf(m, mk);
        }
        shift = -m;
        l = 0.f;
        float inv = 1.f;
        if constexpr (BYTES) {
            for (int k = 0; k < w.n_chunk; ++k) {
                float mk, lk;
                get2(part, k * stride + ml, mk, lk);
                l += lk * join_weight(mk, m);
            }
            inv = inverse_sum(l);
        }
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                o[d][r] = 0.f;
#pragma unroll 1
        for (int k = 0; k < w.n_chunk; ++k) {
            float mk, lk;
            get2(part, k * stride + ml, mk, lk);
            const float f = BYTES ? lk * join_weight(mk, m) * inv : join_weight(mk, m);
            af4 x[DT][4];
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    x[d][r] = get4(part, k * stride + row + 32 * d + 8 * r);
            if constexpr (!BYTES)
                l += lk * f;
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    o[d][r] += x[d][r / 4][r % 4] * f;
        }
    }
    if (live) {
        const float inv = BYTES ? 1.f : inverse_sum(l);
        const int64_t at = (int64_t)(p.row0 + tok) * a.nq + head;
        float *row = a.o + at * D + 4 * hf;
        float2 own = make_float2(0.f, 0.f);
        if constexpr (SHARED)
            own = *reinterpret_cast<const float2 *>(a.stats + 2 * at);
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                af4 *out = reinterpret_cast<af4 *>(row + 32 * d + 8 * r);
                const af4 x = af4{o[d][4 * r] * inv, o[d][4 * r + 1] * inv, o[d][4 * r + 2] * inv, o[d][4 * r + 3] * inv};
                if constexpr (SHARED)
                    *out = join_means(x, -shift, l, *out, own.x, own.y);
                else
                    *out = x;
            }
    }
}

// Rows of a split tile from its partial results.  A workgroup takes four rows of a tile and KV head at a
// time; a thread four channels of a row and every `parts`-th split, in order, then the parts are added
// in order.
// MEANS: the parts are means.  SHARED: joined with what is in o and stats (all tiles are split).
template <bool MEANS, bool SHARED>
__global__ __launch_bounds__(256) void k_attn_prompt_join(AttnArgs a)
{
    __shared__ __attribute__((aligned(16))) af4 s_sum[256];
    __shared__ float s_m[256], s_l[256];
    if ((int)blockIdx.x >= *a.pairs)
        return;
    const PromptSplit p = a.splits[blockIdx.x];
    const int splits = p.n_chunk;
    if (!SHARED && splits <= 1)
        return;
    const int D = a.c.hd, lanes = D / 4, items = 4 * lanes, parts = 256 / items;
    const int tid = threadIdx.x, e = tid % items, k0 = tid / items, row = e / lanes, d4 = e % lanes;
    const int64_t stride = prompt_part_floats(D);
    for (int r0 = 4 * blockIdx.y; r0 < PT_ROWS && (p.rho0 + r0) / a.group < p.rows; r0 += 4 * gridDim.y) {
        const float *part = a.part + p.slot0 * stride, *from = part + (r0 + row) * D + 4 * d4;
        const float *ml = part + PT_ROWS * D + 2 * (r0 + row);
        float m = -INFINITY, l = 0.f, all_m = 0.f, all_l = 0.f;
        af4 sum = {0.f, 0.f, 0.f, 0.f};
        if constexpr (MEANS) {
            // the factors of all parts first, then each mean by its own: threads of a row add them alike
            for (int kb = 0; kb < splits; kb += 8) {
                float2 w[8];
#pragma unroll
                for (int x = 0; x < 8; ++x)                    // all loads in flight at once
                    w[x] = *reinterpret_cast<const float2 *>(ml + min(kb + x, splits - 1) * stride);
                float mb = m;
#pragma unroll
                for (int x = 0; x < 8; ++x)
                    mb = fmaxf(mb, w[x].x);
                l *= join_weight(m, mb);
                m = mb;
#pragma unroll
                for (int x = 0; x < 8; ++x)
                    if (kb + x < splits)
                        l += w[x].y * join_weight(w[x].x, m);
            }
            const float inv = inverse_sum(l);
            all_m = m;
            all_l = l;
            for (int kb = k0; k0 < parts && kb < splits; kb += 8 * parts) {
                af4 v[8];
                float2 w[8];
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    const int64_t at = min(kb + x * parts, splits - 1) * stride;
                    w[x] = *reinterpret_cast<const float2 *>(ml + at);
                    v[x] = *reinterpret_cast<const af4 *>(from + at);
                }
#pragma unroll
                for (int x = 0; x < 8; ++x)
                    if (kb + x * parts < splits)
                        sum += v[x] * (w[x].y * join_weight(w[x].x, m) * inv);
            }
            l = 1.f / parts;                           // the parts' sums are added as they are
            m = 0.f;
        } else {
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
                m = all;
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
        if (k0 == 0 && tok < p.rows) {
            const int64_t at = (int64_t)(p.row0 + tok) * a.nq + p.hkv * a.group + rho % a.group;
            af4 *out = reinterpret_cast<af4 *>(a.o + at * D + 4 * d4);
            const af4 mean = sum * inverse_sum(l);
            if constexpr (SHARED) {
                const float2 own = *reinterpret_cast<const float2 *>(a.stats + 2 * at);
                *out = join_means(mean, MEANS ? all_m : m, MEANS ? all_l : l, *out, own.x, own.y);
            } else {
                *out = mean;
            }
        }
    }
}

}  // namespace qg
