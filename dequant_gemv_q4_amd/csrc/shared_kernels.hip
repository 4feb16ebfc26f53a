// shared_kernels.hip -- attention of a batch whose sequences begin alike, by 16-column tiles: the shared positions
// and those behind them side by side in one launch (attn_shared.h).
#include <hip/hip_runtime.h>

#include "attn8_impl.h"
#include "attn_impl.h"

namespace qg {

// The first `lead` workgroups take the shared positions (g: the groups as sequences of rows), the others what is
// behind them.
template <int T, int D>
__global__ __launch_bounds__(256, D <= 128 ? 2 : 1) void k_shared_16(AttnArgs a, AttnArgs g, int lead, int slots)
{
    const int id = blockIdx.x, behind_them = (int)gridDim.x - lead;
    if constexpr (kv_bytes(T)) {
        __shared__ Attn8Lds<T, D> sh;
        if (id < lead)
            attn8_body<T, D, PREFIX, true>(g, lead, id, lead, sh);
        else
            attn8_body<T, D, SUFFIX, false>(a, slots, id - lead, behind_them, sh);
    } else {
        __shared__ AttnLds<T, D> sh;
        if (id < lead)
            attn_body<T, D, PREFIX, true>(g, lead, id, lead, sh);
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

SharedForm shared_form(int64_t n_seq, int n_group, int nq, int nkv, int hd, int64_t positions)
{
    if (n_seq * nq <= MEET_MOST && prompt_in_16s(n_seq, n_group, nq, nkv, hd, positions))
        return SHARED_16;
    const PromptPlan p = plan_prompt(n_seq, n_group, nkv, nq / nkv, hd, positions);
    return p.pairs < prompt_slots(hd) ? SHARED_PARTED : p.slots ? SHARED_FEW : SHARED_WHOLE;
}

int launch_shared_16(int kv_type, const AttnArgs &a, void *stream)
{
    // slots for either half: what is behind the prefix takes what it can fill, up to a half
    const int all = attn_slots(a.c.hd);
    const int64_t pairs = (int64_t)a.c.n_seq * a.c.nkv * ((a.group + 15) / 16);
    const int slots = (int)(pairs < all / 2 ? pairs : all / 2), lead = all - slots;
    const int64_t table = (int64_t)a.c.max_pages << a.c.ps_log2;
    const bool split = table > (kv_bytes(kv_type) ? Attn8Cols::SOLO << Attn8Cols::UNIT_LOG2
                                                  : AttnCols::SOLO << AttnCols::UNIT_LOG2);
    const int64_t grid = lead + pairs + (split ? slots : 0);
    const AttnArgs g = groups_of(a);
    void (*k)(AttnArgs, AttnArgs, int, int) = nullptr;
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
    hipLaunchKernelGGL(k, dim3((unsigned)grid), dim3(256), 0, static_cast<hipStream_t>(stream), a, g, lead, slots);
    return (int)hipGetLastError();
}

int launch_attn_shared(int kv_type, const AttnArgs &a, void *stream)
{
    const int64_t table = (int64_t)a.c.max_pages << a.c.ps_log2;
    return shared_form(a.c.n_seq, a.n_group, a.nq, a.c.nkv, a.c.hd, table) == SHARED_16
               ? launch_shared_16(kv_type, a, stream)
               : launch_shared_128(kv_type, a, stream);
}

}  // namespace qg
