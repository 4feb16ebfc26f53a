// shared_prompt_kernels.hip -- attention of a batch whose sequences begin alike, the shared positions by 128-column
// tiles of a group's rows.
#include <hip/hip_runtime.h>

#include "attn8_impl.h"
#include "attn_impl.h"
#include "attn_prompt_impl.h"

namespace qg {

template <int T, int D>
__device__ __forceinline__ void tail_body(const AttnArgs &a, int id, int grid, uint8_t *lds)
{
    if constexpr (kv_bytes(T))
        attn8_body<T, D, TAIL, false>(a, attn_slots(D), id, grid, *reinterpret_cast<Attn8Lds<T, D> *>(lds));
    else
        attn_body<T, D, TAIL, false>(a, attn_slots(D), id, grid, *reinterpret_cast<AttnLds<T, D> *>(lds));
}
template <int T, int D>
constexpr size_t tail_lds()
{
    if constexpr (kv_bytes(T))
        return sizeof(Attn8Lds<T, D>);
    else
        return sizeof(AttnLds<T, D>);
}

// What is behind the prefix, alone.
template <int T, int D>
__global__ __launch_bounds__(256, D <= 128 ? 2 : 1) void k_tail(AttnArgs a)
{
    __shared__ __attribute__((aligned(16))) uint8_t lds[tail_lds<T, D>()];
    tail_body<T, D>(a, blockIdx.x, gridDim.x, lds);
}

// As many tiles as slots: those longer than the rest are split (FEW) or none, joined with what k_tail left.
template <int T, int D, bool FEW>
__global__ __launch_bounds__(256, D <= 128 ? 2 : 1) void k_shared_tiles(AttnArgs g, int slots)
{
    __shared__ PromptLds<T, D> sh;
    prompt_body<T, D, FEW, JOINED>(g, slots, blockIdx.x, sh);
}

// Fewer tiles than slots: their parts (the first `slots` workgroups) and what is behind the prefix side by side.
template <int T, int D>
__global__ __launch_bounds__(256, D <= 128 ? 2 : 1) void k_shared_128(AttnArgs a, AttnArgs g, int slots)
{
    constexpr size_t BYTES = sizeof(PromptLds<T, D>) > tail_lds<T, D>() ? sizeof(PromptLds<T, D>) : tail_lds<T, D>();
    __shared__ __attribute__((aligned(1024))) uint8_t lds[BYTES];
    const int id = blockIdx.x;
    if (id < slots)
        prompt_body<T, D, false, PARTED>(g, slots, id, *reinterpret_cast<PromptLds<T, D> *>(lds));
    else
        tail_body<T, D>(a, id - slots, (int)gridDim.x - slots, lds);
}

int launch_shared_128(int kv_type, const AttnArgs &a, void *stream)
{
    hipStream_t s = static_cast<hipStream_t>(stream);
    const bool bytes = kv_bytes(kv_type);
    const int64_t table = (int64_t)a.c.max_pages << a.c.ps_log2;
    AttnArgs g = a;
    g.c.q_start = a.group_start;
    g.c.n_seq = a.n_group;
    const PromptPlan p = plan_prompt(g.c.n_rows, g.c.n_seq, g.c.nkv, g.group, g.c.hd, table);
    const int64_t pairs = (int64_t)a.c.n_seq * a.c.nkv * ((a.group + 15) / 16);
    const int all = attn_slots(a.c.hd);
    const bool split = table > (bytes ? Attn8Cols::SOLO << Attn8Cols::UNIT_LOG2 : AttnCols::SOLO << AttnCols::UNIT_LOG2);
    const int64_t tails = pairs < all ? (split ? all : pairs) : split ? pairs + all : pairs;
    const SharedForm form = shared_form(kv_type, a.c.n_seq, a.n_group, a.nq, a.c.nkv, a.c.hd, table);
    if (form == SHARED_PARTED) {
        void (*k)(AttnArgs, AttnArgs, int) = nullptr;
#define QG_SHARED_D(DD)                                  \
    k = kv_type == KV_F16    ? k_shared_128<KV_F16, DD>  \
        : kv_type == KV_BF16 ? k_shared_128<KV_BF16, DD> \
        : kv_type == KV_I8   ? k_shared_128<KV_I8, DD>   \
                             : k_shared_128<KV_F8, DD>
        switch (a.c.hd) {
        case 64: QG_SHARED_D(64); break;
        case 96: QG_SHARED_D(96); break;
        case 128: QG_SHARED_D(128); break;
        case 192: QG_SHARED_D(192); break;
        default: QG_SHARED_D(256); break;
        }
#undef QG_SHARED_D
        const int slots = bytes && a.c.hd <= 128 ? SHARED_SLOTS_8 : SHARED_SLOTS;
        hipLaunchKernelGGL(k, dim3((unsigned)(slots + tails)), dim3(256), 0, s, a, g, slots);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return (int)e;
        const int64_t share = 4096 / p.pairs;
        const unsigned y = (unsigned)(share > PT_ROWS / 4 ? PT_ROWS / 4 : share > 8 ? share : 8);
        auto join = bytes ? k_attn_prompt_join<true, true> : k_attn_prompt_join<false, true>;
        hipLaunchKernelGGL(join, dim3((unsigned)p.pairs, y), dim3(256), 0, s, g);
        return (int)hipGetLastError();
    }
    void (*t)(AttnArgs) = nullptr;
    void (*k)(AttnArgs, int) = nullptr;
#define QG_SHARED_T(T, DD) (t = k_tail<T, DD>, form == SHARED_FEW ? k_shared_tiles<T, DD, true> : k_shared_tiles<T, DD, false>)
#define QG_SHARED_D(DD)                                 \
    k = kv_type == KV_F16    ? QG_SHARED_T(KV_F16, DD)  \
        : kv_type == KV_BF16 ? QG_SHARED_T(KV_BF16, DD) \
        : kv_type == KV_I8   ? QG_SHARED_T(KV_I8, DD)   \
                             : QG_SHARED_T(KV_F8, DD)
    switch (a.c.hd) {
    case 64: QG_SHARED_D(64); break;
    case 96: QG_SHARED_D(96); break;
    case 128: QG_SHARED_D(128); break;
    case 192: QG_SHARED_D(192); break;
    default: QG_SHARED_D(256); break;
    }
#undef QG_SHARED_D
#undef QG_SHARED_T
    hipLaunchKernelGGL(t, dim3((unsigned)tails), dim3(256), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return (int)e;
    const int few = form == SHARED_FEW ? p.slots : 0;
    hipLaunchKernelGGL(k, dim3((unsigned)(p.pairs + few)), dim3(256), 0, s, g, few);
    return (int)hipGetLastError();
}

}  // namespace qg
