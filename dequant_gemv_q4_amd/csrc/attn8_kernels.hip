// attn8_kernels.hip -- attention of one or a few new rows per sequence over 8-bit pages (attn8_impl.h).
#include <hip/hip_runtime.h>

#include "attn8_impl.h"

namespace qg {

template <int T, int D, int FORM, bool SIDE>
__global__ __launch_bounds__(256, D <= 128 ? 2 : 1) void k_attn8(AttnArgs a)
{
    __shared__ Attn8Lds<T, D> sh;
    attn8_body<T, D, FORM, SIDE>(a, attn_slots(D), blockIdx.x, gridDim.x, sh);
}

template <int FORM>
static int launch_k_attn8(int kv_type, const AttnArgs &a, int64_t pairs, void *stream)
{
    const int slots = attn_slots(a.c.hd);
    void (*k)(AttnArgs) = nullptr;
#define QG_ATTN8_T(T, DD) \
    a.side > 1 ? k_attn8<T, DD, FORM, true> : k_attn8<T, DD, FORM, false>
#define QG_ATTN8_D(DD) k = kv_type == KV_I8 ? QG_ATTN8_T(KV_I8, DD) : QG_ATTN8_T(KV_F8, DD)
    switch (a.c.hd) {
    case 64: QG_ATTN8_D(64); break;
    case 96: QG_ATTN8_D(96); break;
    case 128: QG_ATTN8_D(128); break;
    case 192: QG_ATTN8_D(192); break;
    default: QG_ATTN8_D(256); break;
    }
#undef QG_ATTN8_D
#undef QG_ATTN8_T
    // as many pairs as slots: those that are much longer than the rest are split all the same
    const int64_t table = (int64_t)a.c.max_pages << a.c.ps_log2;
    const int64_t grid = pairs < slots ? slots : table > Attn8Cols::SOLO << Attn8Cols::UNIT_LOG2 ? pairs + slots : pairs;
    hipLaunchKernelGGL(k, dim3((unsigned)grid), dim3(256), 0, static_cast<hipStream_t>(stream), a);
    return (int)hipGetLastError();
}

int launch_attn8(int kv_type, const AttnArgs &a, void *stream)
{
    AttnArgs b = a;
    b.side = (a.group + 15) / 16;
    return launch_k_attn8<ONE>(kv_type, b, (int64_t)a.c.n_seq * a.c.nkv * b.side, stream);
}

int launch_attn8_rows(int kv_type, const AttnArgs &a, void *stream)
{
    AttnArgs b = a;
    b.side = (int)((a.c.n_rows * a.group + 16 * a.c.n_seq - 1) / (16 * a.c.n_seq));   // on average
    return launch_k_attn8<MANY>(kv_type, b, a.c.nkv * (a.c.n_rows * a.group / 16 + a.c.n_seq), stream);
}

}  // namespace qg
