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
// operands: two f16 hold 22 of its 24 bits down to 2^-3 (below that, 2^-25 is lost), three bf16 all of
// them.  (Two bf16, 2^-18, left attention outputs 2.4e-6 off in the root mean square where f32 sums leave
// 0.7e-6.)
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

// The weight of a score s (in powers of two) is held as 2^(s + shift).  A row's shift is LIFT less the
// largest score it has seen, until a later one would bring the exponent above TOP: then it moves (a wave
// vote, so that the accumulators are rescaled a few times in a row's life).  f16 ends at 2^16 and loses
// what is below 2^-25, so of weights far below the largest one 2^-25 / 2^10 = 2^-35 of it is lost at most.
// (With LIFT 6, 2^-31 of it: one position with 90 % of the weight and a hundredth of the others' values
// before 8191 others, outputs 2.3e-6 off in the root mean square; 1.07e-6 with 10, and 1.06e-6 with bf16's
// 24 bits.)  A LIFT nearer to TOP rescales more often: three prompts of 1310 rows in all (14 / 2 heads of
// 256) 42.9 us with 6 and 13, 42.4 with these, 45.0 with 12.  bf16 has f32's range, so its weights are at
// most 1: with V up to the type's end their products stay within f32.
template <int T> constexpr float LIFT = T == KV_F16 ? 10.0f : -7.0f;
template <int T> constexpr float TOP = T == KV_F16 ? 15.9f : 0.0f;
// No score yet: any score moves it, and a masked one (-inf) weighs 0.
constexpr float NO_SHIFT = 3.402823466e38f;
// Scores beyond 2^24 are more than 2 apart, and LIFT less one of them is rounded to such steps: where that
// would end above TOP, 0 is as good for weights that are steps of 2^-8 apart.
template <int T>
__device__ __forceinline__ float shift_of(float top_score)
{
    const float r = LIFT<T> - top_score;
    return r + top_score > TOP<T> ? -top_score : r;
}

// Joining partial results (O, exponent m = -shift, sum) of parts of the positions: each O and sum is
// weighted by join_weight with the largest m, whatever it is, and the whole divided by the sum.  A part in
// which a row sees nothing has zeros and the lowest m.  So does, as to m, one in which it sees only NaN
// scores (fmaxf passes NaN over), and a part with some may weigh 0; their sums are NaN and stay so, as 0 x
// NaN is NaN: no part may be left out for its m or its weight.
__device__ __forceinline__ float join_weight(float part_m, float largest_m)
{
    return part_m == largest_m ? 1.0f : __builtin_amdgcn_exp2f(part_m - largest_m);
}
// 1 / sum, or 0 for a row that sees nothing.
__device__ __forceinline__ float inverse_sum(float l) { return l == 0.f ? 0.f : 1.0f / l; }

// Partial results that pass between workgroups of one launch, which may run on different XCDs: every
// access carries the agent-scope bit (sc1), so that it neither stays in nor is answered by the L2 of one
// XCD.  Offsets in floats.
constexpr int AGENT_SCOPE = 16;                           // the buffer instructions' sc1
typedef uint32_t au2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ void put4(__amdgpu_buffer_rsrc_t r, uint32_t at, af4 v)
{
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(au4, v), r, 4 * at, 0, AGENT_SCOPE);
}
__device__ __forceinline__ af4 get4(__amdgpu_buffer_rsrc_t r, uint32_t at)
{
    return __builtin_bit_cast(af4, __builtin_amdgcn_raw_buffer_load_b128(r, 4 * at, 0, AGENT_SCOPE));
}
__device__ __forceinline__ void put2(__amdgpu_buffer_rsrc_t r, uint32_t at, float a, float b)
{
    const au2 v = {__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b)};
    __builtin_amdgcn_raw_buffer_store_b64(v, r, 4 * at, 0, AGENT_SCOPE);
}
__device__ __forceinline__ void get2(__amdgpu_buffer_rsrc_t r, uint32_t at, float &a, float &b)
{
    const au2 v = __builtin_amdgcn_raw_buffer_load_b64(r, 4 * at, 0, AGENT_SCOPE);
    const uint32_t v0 = v[0], v1 = v[1];
    a = __builtin_bit_cast(float, v0);
    b = __builtin_bit_cast(float, v1);
}

// Whether this workgroup is the last of `members` to arrive at a counter (left at 0 by the last).
// Its partial results are complete in memory before it arrives: each wave waits for its own stores
// (vmcnt counts an agent-scope store until it is done), then the workgroup meets.
__device__ __forceinline__ bool last_to_arrive(unsigned int *cnt, int members, int *s_last)
{
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (threadIdx.x == 0) {
        const unsigned int before =
            __hip_atomic_fetch_add(cnt, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        *s_last = before + 1 == (unsigned int)members;
        if (*s_last)
            __hip_atomic_store(cnt, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    asm volatile("" ::: "memory");
    return *s_last != 0;
}

// ------------------------------------------------------------- work of a call, from lengths on the device
//
// The new rows of a sequence times the query heads of a KV head are columns rho = token * group +
// head; a workgroup takes COLS of them (a pair: sequence and KV head, tile of columns) against a
// chunk of the sequence's positions.  The lengths are on the device, so every workgroup derives the
// same plan from them: where there are fewer pairs than workgroup slots, the smallest chunk (whole
// units of 2^UNIT_LOG2 positions, at least LEAST) for which the chunks of all pairs fit the slots; a
// pair's chunks are equal to one unit.  With as many pairs as slots only the longest are split.  Sequences
// of up to SOLO units are not split, those of up to FLAT units into at most RADIX chunks.  INDEX: the plan
// also numbers the pairs and, with as many as slots, puts the longest of those that are not split first.
// SIDE: a KV head's tiles that read the same chunk come side by side, not each tile's chunks.
template <int COLS_, int UNIT_LOG2_, int LEAST_, int SOLO_, int FLAT_, int RADIX_, bool INDEX_, bool SIDE_>
struct PlanOf {
    static constexpr int COLS = COLS_, UNIT_LOG2 = UNIT_LOG2_, LEAST = LEAST_, SOLO = SOLO_;
    static constexpr int FLAT = FLAT_, RADIX = RADIX_;
    static_assert(RADIX >= 1, "a sequence without positions has a chunk");
    static constexpr bool INDEX = INDEX_, SIDE = SIDE_;
    static __device__ __forceinline__ int units(int n) { return (n + (1 << UNIT_LOG2) - 1) >> UNIT_LOG2; }
    // at least one, so that an empty sequence's rows are written
    static __device__ __forceinline__ int chunks(int n, int u)
    {
        const int x = units(n);
        const int n_chunk = x <= u || x <= SOLO ? 1 : (x + u - 1) / u;
        return x <= FLAT && n_chunk > RADIX ? RADIX : n_chunk;
    }
};

struct AttnPlan {
    int b, pair, chunk, n_chunk;   // this workgroup's sequence, pair within it, chunk of its chunks
    int slot0;                     // slot of the pair's first chunk
    int first_pair, pairs;         // pairs of earlier sequences (where INDEX and all), of all
    bool all;                      // fewer pairs than slots: all of them share the slots
    int len;                       // the sequence's positions
    int row0, rows;                // its new rows
};

// What the plan has to know of a sequence.
struct AttnSeq {
    int n, pairs, row0, rows;
};

// Positions of sequence b that have a place in its table.
__device__ __forceinline__ int seq_len(const KvArgs &c, int b)
{
    const int n = c.kv_len[b], cap = c.max_pages << c.ps_log2;          // cap <= 2^24
    if (n > cap)
        atomicOr(c.err, 1u);
    return n < 0 ? 0 : n < cap ? n : cap;
}

// First new row of sequence i, cut to the rows there are.
__device__ __forceinline__ int row_start(const KvArgs &c, int i)
{
    const int64_t v = c.q_start[i];
    return (int)(v < 0 ? 0 : v < c.n_rows ? v : c.n_rows);
}

// Inclusive sum (or f, with f(v, 0) = v) over the lanes up to this one; lane 63 has the total.
template <class F>
__device__ __forceinline__ int wave_scan(int v, F f)
{
    v = f(v, __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true));      // row_shr 1, 2, 4, 8
    v = f(v, __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true));
    v = f(v, __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true));
    v = f(v, __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true));
    v = f(v, __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false));     // row 0 -> 1, 2 -> 3
    v = f(v, __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false));     // rows 0, 1 -> 2, 3
    return v;
}
__device__ __forceinline__ int wave_scan(int v)
{
    return wave_scan(v, [](int a, int b) { return a + b; });
}
__device__ __forceinline__ int wave_sum(int v) { return __builtin_amdgcn_readlane(wave_scan(v), 63); }
__device__ __forceinline__ int wave_top(int v)          // v >= 0
{
    return __builtin_amdgcn_readlane(wave_scan(v, [](int a, int b) { return a > b ? a : b; }), 63);
}

// The id-th pair of an unsplit plan in falling order of work, so that the workgroups that start last are
// short and all end together.  Tile x of a sequence counts x + 1 and the tiles that its earlier positions
// would fill; the counts are cut into up to LEVELS levels (a binary search of six steps), within a level
// the pairs go by sequence.  Against sequence after sequence: nine prompts, 4500 rows (24 / 8 heads of 64,
// bf16) 40.0 -> 36.5 us; five, 2000 rows (32 / 8 of 128, bf16) 47.0 -> 39.1; a hundred, 8000 rows behind up
// to 500 positions (12 / 2 of 128) 59.3 -> 51.5; two of 2000 (8 / 8 of 256) 68.0 -> 67.8; three, 4000 rows
// behind up to 8000 (32 / 8 of 128) 621 -> 635.
template <class P, class Seq>
__device__ __forceinline__ bool longest_first(const KvArgs &c, int n_seq, int group, int id, AttnPlan &p, Seq seq)
{
    constexpr int LEVELS = 64;
    auto behind = [&](const AttnSeq &s) { return (int)((int64_t)max(s.n - s.rows, 0) * group / P::COLS); };
    auto tiles = [&](const AttnSeq &s) { return (int)(((int64_t)s.rows * group + P::COLS - 1) / P::COLS); };
    int top = 0;
    for (int b0 = 0; b0 < n_seq; b0 += 64) {
        const AttnSeq s = seq(b0);
        top = max(top, tiles(s) + behind(s));
    }
    top = wave_top(top);
    const int step = top / LEVELS + 1;
    // tiles of a sequence at a level or above
    auto from = [&](const AttnSeq &s, int level) {
        const int t = tiles(s);
        return min(max(t + behind(s) + 1 - level * step, 0), t);
    };
    auto pairs_from = [&](int level) {
        int v = 0;
        for (int b0 = 0; b0 < n_seq; b0 += 64)
            v += from(seq(b0), level);
        return c.nkv * wave_sum(v);
    };
    int lo = 0, hi = top / step;
    while (lo < hi) {
        const int mid = lo + (hi - lo + 1) / 2;
        if (pairs_from(mid) > id)
            lo = mid;
        else
            hi = mid - 1;
    }
    int base = pairs_from(lo + 1);
    for (int b0 = 0; b0 < n_seq; b0 += 64) {
        const AttnSeq s = seq(b0);
        const int above = from(s, lo + 1), here = c.nkv * (from(s, lo) - above), end = base + wave_scan(here);
        const uint64_t in = __ballot(id < end);
        if (in) {
            const int l = __ffsll((unsigned long long)in) - 1;
            const int r = id - __builtin_amdgcn_readlane(end - here, l);
            const int x = __builtin_amdgcn_readlane(tiles(s) - 1 - above, l) - r / c.nkv;
            p.b = b0 + l;
            p.pair = x * c.nkv + r % c.nkv;
            p.chunk = p.slot0 = 0;
            p.n_chunk = 1;
            p.len = __builtin_amdgcn_readlane(s.n, l);
            p.row0 = __builtin_amdgcn_readlane(s.row0, l);
            p.rows = __builtin_amdgcn_readlane(s.rows, l);
            // (row starts that are not in order could give sums beyond an int)
            return r >= 0 && x >= 0;
        }
        base = __builtin_amdgcn_readlane(end, 63);
    }
    return false;
}

// Units of the longest sequence and of all pairs (up to 2^41, in two halves).
struct AttnTotals {
    int longest, low, high;
    template <class P> __device__ __forceinline__ void add(const AttnSeq &s)
    {
        const int n = P::units(s.n);
        const int64_t v = (int64_t)s.pairs * n;
        longest = max(longest, s.pairs ? n : 0);
        low += (int)(v & 0xFFF);
        high += (int)(v >> 12);
    }
    __device__ __forceinline__ AttnTotals of_wave() const
    {
        return {wave_top(longest), wave_sum(low), wave_sum(high)};
    }
};

// The plan from the sequences `seq(b0)` of lanes b0 .. b0 + 63 of each round.
template <class P, bool ROWS, class Seq, class Totals>
__device__ __forceinline__ bool attn_plan_of(const KvArgs &c, int n_seq, int group, int slots, bool all, int id,
                                             AttnPlan &p, Seq seq, Totals totals)
{
    auto sum = [&](auto of) {
        int v = 0;
        for (int b0 = 0; b0 < n_seq; b0 += 64)
            v += of(seq(b0));
        return wave_sum(v);
    };
    int u = 0x3fffffff;
    bool some = false, whole = false;                  // some pairs are split; this is one of those that are not
    p.pairs = ROWS ? sum([](const AttnSeq &s) { return s.pairs; })
                   : c.n_seq * c.nkv * ((group + P::COLS - 1) / P::COLS);
    p.all = all && p.pairs >= 0 && p.pairs < slots;
    if (p.all) {
        // chunks <= units / u + 1 each, so u = units / (slots - pairs), over all pairs, is enough;
        // units / slots is the least that could be
        const int units = sum([](const AttnSeq &s) { return s.pairs * P::units(s.n); });
        int lo = max((units + slots - 1) / slots, P::LEAST);
        int hi = max((units + slots - p.pairs - 1) / (slots - p.pairs), lo);
        while (lo < hi) {
            const int mid = lo + (hi - lo) / 2;
            if (sum([=](const AttnSeq &s) { return s.pairs * P::chunks(s.n, mid); }) <= slots)
                hi = mid;
            else
                lo = mid + 1;
        }
        u = lo;
    } else if (slots && p.pairs > 0 && !(P::INDEX && all)) {
        // As many pairs as slots: only those of more units than a slot's share are split (their chunks
        // come first), as far as their parts fit the slots; at twice the share they do.  64 sequences of
        // one token, the longest of 20000 positions (32 / 8 heads of 128): unsplit 286 us, 184; of 10000
        // (8 / 8 of 64) 107 and 61; 256 of about 1100 (12 / 2), where none is split, 58.1 and 58.2.
        const AttnTotals t = totals();
        const int share = (int)((((int64_t)t.high << 12) + t.low + slots - 1) / slots);
        int lo = max(share, max(P::LEAST, P::SOLO)), hi = max(2 * share, lo);
        if (t.longest > lo) {
            auto split_at = [&](int v) {
                return sum([=](const AttnSeq &s) { return P::chunks(s.n, v) > 1 ? s.pairs * P::chunks(s.n, v) : 0; });
            };
            while (lo < hi) {
                const int mid = lo + (hi - lo) / 2;
                if (split_at(mid) <= slots)
                    hi = mid;
                else
                    lo = mid + 1;
            }
            u = lo;
            const int split = split_at(u);
            some = true;
            whole = id >= split;
            id -= whole ? split : 0;
        }
    }
    if (P::INDEX && !p.all && (whole || !some)) {
        if (id >= p.pairs)
            return false;
        if (c.n_seq > 1)
            return longest_first<P>(c, n_seq, group, id, p, [&](int b0) {
                AttnSeq s = seq(b0);
                const bool mine = !some || P::chunks(s.n, u) == 1;
                s.n = mine ? s.n : 0;
                s.rows = mine ? s.rows : 0;
                return s;
            });
        id = p.pairs - 1 - id;
    }
    if (!P::INDEX && !ROWS && !p.all && !some) {           // every sequence has the same pairs
        const int per = c.nkv * ((group + P::COLS - 1) / P::COLS);
        p.b = id / per;
        if (p.b >= c.n_seq)
            return false;
        const AttnSeq s = seq(p.b & ~63);
        p.pair = id % per;
        p.chunk = p.slot0 = 0;
        p.n_chunk = 1;
        p.len = __builtin_amdgcn_readlane(s.n, p.b & 63);
        p.row0 = p.b;
        p.rows = 1;
        return true;
    }
    int base = 0, before = 0;
    for (int b0 = 0; b0 < n_seq; b0 += 64) {
        const AttnSeq s = seq(b0);
        int nc = P::chunks(s.n, u);
        if (some)
            nc = whole == (nc == 1) ? nc : 0;
        const int end = base + wave_scan(nc * s.pairs);
        const int pe = P::INDEX ? before + wave_scan(s.pairs) : 0;
        const uint64_t in = __ballot(id < end);
        if (in) {
            const int l = __ffsll((unsigned long long)in) - 1;
            p.b = b0 + l;
            p.n_chunk = __builtin_amdgcn_readlane(nc, l);
            p.len = __builtin_amdgcn_readlane(s.n, l);
            p.slot0 = __builtin_amdgcn_readlane(end - nc * s.pairs, l);
            p.first_pair = P::INDEX ? __builtin_amdgcn_readlane(pe - s.pairs, l) : 0;
            p.row0 = ROWS ? __builtin_amdgcn_readlane(s.row0, l) : p.b;
            p.rows = ROWS ? __builtin_amdgcn_readlane(s.rows, l) : 1;
            const int pairs = __builtin_amdgcn_readlane(s.pairs, l), r = id - p.slot0;
            if (!P::SIDE) {
                p.pair = r / p.n_chunk;
                p.chunk = r - p.pair * p.n_chunk;
            } else {
                const int tiles = pairs / c.nkv, head = r / (tiles * p.n_chunk), x = r - head * tiles * p.n_chunk;
                p.chunk = x / tiles;
                p.pair = head * tiles + x - p.chunk * tiles;
            }
            p.slot0 += p.pair * p.n_chunk;
            // (row starts that are not in order could give sums beyond an int)
            return !ROWS || (p.pair >= 0 && p.pair < pairs && p.chunk >= 0 &&
                             (p.n_chunk == 1 || (p.slot0 >= 0 && p.slot0 + p.n_chunk <= slots)));
        }
        base = __builtin_amdgcn_readlane(end, 63);
        before = P::INDEX ? __builtin_amdgcn_readlane(pe, 63) : 0;
    }
    return false;
}

// Workgroup id -> its place in the plan; false if the plan has fewer workgroups.  All threads of the
// workgroup call it; every wave finds the same.  Up to 64 sequences are held a lane each, more in LDS
// scratch (QG_ATTN_MAX_SEQ entries, free again afterwards).  ROWS: sequence b has the rows between its
// q_start and the next; else one row, row b.  slots 0: nothing is split.  INDEX: all pairs
// or only the longest are split, as `all` says.
template <class P, bool ROWS>
__device__ __forceinline__ bool attn_plan(const KvArgs &c, int group, int slots, int id, AttnPlan &p,
                                          AttnSeq *scratch, bool all = true)
{
    const int lane = threadIdx.x & 63;
    auto load = [&](int b) {
        AttnSeq s = {0, 0, b, 0};
        if (b < c.n_seq) {
            s.n = seq_len(c, b);
            s.rows = 1;
            if constexpr (ROWS) {
                s.row0 = row_start(c, b);
                s.rows = max(row_start(c, b + 1) - s.row0, 0);
            }
            s.pairs = c.nkv * (int)(((int64_t)s.rows * group + P::COLS - 1) / P::COLS);
        }
        return s;
    };
    if (c.n_seq <= 64) {
        const AttnSeq s = load(lane);
        return attn_plan_of<P, ROWS>(c, 1, group, slots, all, id, p, [&](int) { return s; }, [&]() {
            AttnTotals t = {0, 0, 0};
            t.add<P>(s);
            return t.of_wave();
        });
    }
    __shared__ AttnTotals s_tot[4];
    AttnTotals t = {0, 0, 0};
    for (int b = threadIdx.x; b < (c.n_seq + 63) / 64 * 64; b += 256) {
        const AttnSeq s = load(b);
        scratch[b] = s;
        t.add<P>(s);
    }
    t = t.of_wave();
    if (lane == 0)
        s_tot[threadIdx.x >> 6] = t;
    __syncthreads();
    const bool found = attn_plan_of<P, ROWS>(
        c, c.n_seq, group, slots, all, id, p, [&](int b0) { return scratch[b0 + lane]; }, [&]() {
            AttnTotals v = {0, 0, 0};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                v.longest = max(v.longest, s_tot[w].longest);
                v.low += s_tot[w].low;
                v.high += s_tot[w].high;
            }
            return v;
        });
    __syncthreads();
    return found;
}

}  // namespace qg
