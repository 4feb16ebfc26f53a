// attn_prompt_kernels.hip -- causal attention of packed sequences of new rows (attn_prompt_impl.h).
#include <hip/hip_runtime.h>

#include "attn_prompt_impl.h"

namespace qg {

template <int T, int D, bool FEW>
__global__ __launch_bounds__(256, D <= 128 ? 2 : 1) void k_attn_prompt(AttnArgs a, int slots)
{
    __shared__ PromptLds<T, D> sh;
    prompt_body<T, D, FEW, CAUSAL>(a, slots, blockIdx.x, sh);
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

// The same over 8-bit pages, where the 16-column kernel reads half the bytes and the 128-row tiles convert the codes
// on their way through LDS: resident workgroups and bounded work are enough.  128-row tiles -> 16 columns, us, I8:
// one sequence of 128 rows x 4000, 12 / 2 heads of 128, 40.7 -> 31.1, 32 / 8 heads (2.2e9 channels) 54.1 -> 47.1;
// 64 rows x 20000, 16 / 1, 62.0 -> 54.0, 24 / 8 of 64 48.7 -> 47.7; 128 rows x 20000, 12 / 2 (3.2e9) 64.9 -> 69.7;
// 200 rows x 10000, 24 / 8 of 64 (3.1e9) 58.4 -> 91.1.
bool prompt8_in_16s(int64_t n_rows, int n_seq, int nq, int nkv, int hd, int64_t positions)
{
    return nkv * (n_rows * (nq / nkv) / 16 + n_seq) <= attn_slots(hd) &&
           n_rows * nq * hd * (positions < 16384 ? positions : 16384) <= 2500000000LL;
}

int launch_attn_prompt(int kv_type, const AttnArgs &a, void *stream)
{
    const int64_t table = (int64_t)a.c.max_pages << a.c.ps_log2;
    const bool bytes = kv_bytes(kv_type);
    if ((bytes ? prompt8_in_16s : prompt_in_16s)(a.c.n_rows, a.c.n_seq, a.nq, a.c.nkv, a.c.hd, table))
        return bytes ? launch_attn8_rows(kv_type, a, stream) : launch_attn_rows(kv_type, a, stream);
    hipStream_t s = static_cast<hipStream_t>(stream);
    const PromptPlan p = plan_prompt(a.c.n_rows, a.c.n_seq, a.c.nkv, a.group, a.c.hd, table);
    const bool few = p.slots && !p.second;
    void (*k)(AttnArgs, int) = nullptr;
#define QG_PROMPT_T(T, DD) few ? k_attn_prompt<T, DD, true> : k_attn_prompt<T, DD, false>
#define QG_PROMPT_D(DD)                                 \
    k = kv_type == KV_F16    ? QG_PROMPT_T(KV_F16, DD)  \
        : kv_type == KV_BF16 ? QG_PROMPT_T(KV_BF16, DD) \
        : kv_type == KV_I8   ? QG_PROMPT_T(KV_I8, DD)   \
                             : QG_PROMPT_T(KV_F8, DD)
    switch (a.c.hd) {
    case 64: QG_PROMPT_D(64); break;
    case 96: QG_PROMPT_D(96); break;
    case 128: QG_PROMPT_D(128); break;
    case 192: QG_PROMPT_D(192); break;
    default: QG_PROMPT_D(256); break;
    }
#undef QG_PROMPT_D
#undef QG_PROMPT_T
    hipLaunchKernelGGL(k, dim3((unsigned)p.grid), dim3(256), 0, s, a, p.slots);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !p.second)
        return (int)e;
    // the fewer tiles, the more workgroups share one, about 4096 in all (sixteen sequences of 32 rows
    // behind 4000 positions: 56.3 us, with 2048 61.4; 8192 that find nothing to join cost 1 us more)
    const int64_t share = 4096 / p.pairs;
    const unsigned y = (unsigned)(share > PT_ROWS / 4 ? PT_ROWS / 4 : share > 8 ? share : 8);
    auto join = bytes ? k_attn_prompt_join<true, false> : k_attn_prompt_join<false, false>;
    hipLaunchKernelGGL(join, dim3((unsigned)p.pairs, y), dim3(256), 0, s, a);
    return (int)hipGetLastError();
}

}  // namespace qg
