// shared_kernels.hip -- attention of a batch whose sequences begin alike, by 16-column tiles: the shared positions
// and those behind them side by side in one launch (attn_shared.h).
#include <hip/hip_runtime.h>

#include "attn8_impl.h"
#include "attn_impl.h"

namespace qg {

// The first `lead` workgroups take the shared positions (g: the groups as sequences of rows; `first` slots for a
// split), the others what is behind them (`slots`).
template <int T, int D>
__global__ __launch_bounds__(256, D <= 128 ? 2 : 1) void k_shared_16(AttnArgs a, AttnArgs g, int lead, int first, int slots)
{
    const int id = blockIdx.x, behind_them = (int)gridDim.x - lead;
    if constexpr (kv_bytes(T)) {
        __shared__ Attn8Lds<T, D> sh;
        if (id < lead)
            attn8_body<T, D, PREFIX, true>(g, first, id, lead, sh);
        else
            attn8_body<T, D, SUFFIX, false>(a, slots, id - lead, behind_them, sh);
    } else {
        __shared__ AttnLds<T, D> sh;
        if (id < lead)
            attn_body<T, D, PREFIX, true>(g, first, id, lead, sh);
        else
            attn_body<T, D, SUFFIX, false>(a, slots, id - lead, behind_them, sh);
    }
}

static AttnArgs groups_of(const AttnArgs &a)
{
    AttnArgs g = a;
    g.c.q_start = a.group_start;
    g.c.n_seq = a.n_group;
    g.side = (int)((g.c.n_rows * g.group + 16 * g.c.n_seq - 1) / (16 * g.c.n_seq));   // on average
    return g;
}

// The 16-column tiles read a prefix once per 16 columns, the 128-column ones leave parts for a second launch and
// fill their tiles less.  By the work, columns times positions times channels of all heads (of longer tables 16384
// positions count: a table is sized for the longest cache), at most: over f16 and bf16 pages 5e8, over 8-bit pages,
// whose codes the 128-column tiles convert through LDS, 1.5e9.  16 -> 128 columns, us, 128 channels: f16, 64
// sequences, 32 / 8 heads, behind 1500 positions (4e8) 37.4 -> 37.4, behind 4000 (1.1e9) 46.7 -> 38.3, 30000 (4.3e9)
// 183 -> 93; 12 / 2 heads behind 4000 (4e8) 33.3 -> 34.9, 10000 (1e9) 48.7 -> 37.7; bf16, 150 of 16 / 1 behind 2500
// (8e8) 47.0 -> 42.5; I8, 64 of 32 / 8 behind 4000 (1.1e9) 35.9 -> 43.4, 8000 (2.1e9) 50.0 -> 48.5, 30000 130 -> 111;
// 200 of 12 / 2 behind 4000 (1.3e9) 44.4 -> 43.9, 150 of 16 / 1 behind 2500 (8e8) 38.3 -> 43.7, 10000 (3.1e9) 80.7 ->
// 62.2; heads of 256, 30 of 32 / 8 behind 8000 (2e9) 95.0 -> 78.1; 24 / 8 of 64, 32 behind 20000 (8e8) 36.7 -> 42.7.
// (All with tables as long as the caches; lengths are on the device, so a short prefix in a long table is taken for a
// long one.  Over f16 and bf16 only heads of 128 were timed.)
SharedForm shared_form(int kv_type, int64_t n_seq, int n_group, int nq, int nkv, int hd, int64_t positions)
{
    const double work = (double)(n_seq * nq) * hd * (positions < 16384 ? positions : 16384);
    if (n_seq * nq <= MEET_MOST && work <= (kv_bytes(kv_type) ? 1.5e9 : 5e8))
        return SHARED_16;
    const PromptPlan p = plan_prompt(n_seq, n_group, nkv, nq / nkv, hd, positions);
    return p.pairs < SHARED_SLOTS ? SHARED_PARTED : p.slots ? SHARED_FEW : SHARED_WHOLE;
}

int launch_shared_16(int kv_type, const AttnArgs &a, void *stream)
{
    // Slots for either half.  The prefix leaves to what is behind it a workgroup a pair, up to a half of those that
    // are resident; that half has its slots too, so that long ones are split: two sequences of up to 15000 positions
    // behind 500 (12 / 2 heads of 128, f16) 94 -> 22.5 us in a graph, qgemv_attn 17.7; 16 of 3000 behind 400 (24 / 8 of
    // 64) 26.2 -> 23.4; a prefix of 8000 before 300 of 4 each 23.2 and 23.2 (with half of the slots for it alone 24.4).
    // As many pairs as slots: each has a workgroup, and those that are split as many more as there are slots.
    const int all = attn_slots(a.c.hd);
    const int64_t table = (int64_t)a.c.max_pages << a.c.ps_log2;
    const bool split = table > (kv_bytes(kv_type) ? Attn8Cols::SOLO << Attn8Cols::UNIT_LOG2
                                                  : AttnCols::SOLO << AttnCols::UNIT_LOG2);
    auto grid_of = [=](int64_t pairs, int slots) { return pairs < slots ? slots : pairs + (split ? slots : 0); };
    const int64_t pairs = (int64_t)a.c.n_seq * a.c.nkv * ((a.group + 15) / 16);
    const int few = (int)(pairs < all / 2 ? pairs : all / 2), first = all - few, slots = split ? all / 2 : few;
    const int64_t lead = grid_of(a.c.nkv * (a.c.n_rows * a.group / 16 + a.n_group), first);
    const AttnArgs g = groups_of(a);
    void (*k)(AttnArgs, AttnArgs, int, int, int) = nullptr;
#define QG_SHARED_D(DD)                               \
    k = kv_type == KV_F16    ? k_shared_16<KV_F16, DD>  \
        : kv_type == KV_BF16 ? k_shared_16<KV_BF16, DD> \
        : kv_type == KV_I8   ? k_shared_16<KV_I8, DD>   \
                             : k_shared_16<KV_F8, DD>
    switch (a.c.hd) {
    case 64: QG_SHARED_D(64); break;
    case 96: QG_SHARED_D(96); break;
    case 128: QG_SHARED_D(128); break;
    case 192: QG_SHARED_D(192); break;
    default: QG_SHARED_D(256); break;
    }
#undef QG_SHARED_D
    hipLaunchKernelGGL(k, dim3((unsigned)(lead + grid_of(pairs, slots))), dim3(256), 0, static_cast<hipStream_t>(stream),
                       a, g, (int)lead, first, slots);
    return (int)hipGetLastError();
}

int launch_attn_shared(int kv_type, const AttnArgs &a, void *stream)
{
    const int64_t table = (int64_t)a.c.max_pages << a.c.ps_log2;
    return shared_form(kv_type, a.c.n_seq, a.n_group, a.nq, a.c.nkv, a.c.hd, table) == SHARED_16
               ? launch_shared_16(kv_type, a, stream)
               : launch_shared_128(kv_type, a, stream);
}

}  // namespace qg
