// attn_kernels.hip -- the paged key-value cache: storing new rows, and attention of one new token per
// sequence over it.
#include <hip/hip_runtime.h>

#include "attn_impl.h"

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
// Bound by HBM: 8000 rows of 8 heads of 128 (98.3 MB read and written) take 22.4 us, 4.4 TB/s, where a
// copy reaches 4.94; one position at a time took 75 us.  One row of 2 heads: 2.8 us, a launch.
template <int T, int BL>
__global__ __launch_bounds__(256) void k_kv_append(AppendArgs a)
{
    constexpr int BLOCK = 1 << BL, PIECES_V = BLOCK / 8;
    const KvArgs &c = a.c;
    const int tid = threadIdx.x, h = blockIdx.y;
    int id = blockIdx.x;
    if (c.q_start && c.ps_log2 > BL) {
        // two blocks to an XCD, eight workgroups apart: halves of the same lines of V may meet in its L2
        // (8000 rows, pages of 64: 24.4 -> 23.4 us)
        const int r = id % 16;
        if (id - r + 16 <= (int)gridDim.x)
            id += r % 8 * 2 + r / 8 - r;
    }
    AppendBlock w;
    if (!append_block<BL>(c, id, w))
        return;
    const int page = append_page(c, w);
    if (page < 0) {
        if (tid == 0 && h == 0)
            atomicOr(c.err, 1u);
        return;
    }
    const int64_t t0 = w.t0;
    const int from = w.from, to = w.to;
    // row of position t0 + t at src + t * stride
    const int64_t at = w.row0 * a.stride + (int64_t)h * c.hd;
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

// ---------------------------------------------------- one or a few new rows per sequence (attn_impl.h)

template <int T, int D, int FORM, bool SIDE>
__global__ __launch_bounds__(256, D <= 128 ? 2 : 1) void k_attn(AttnArgs a)
{
    __shared__ AttnLds<T, D> sh;
    attn_body<T, D, FORM, SIDE>(a, attn_slots(D), blockIdx.x, gridDim.x, sh);
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

template <int FORM>
static int launch_k_attn(int kv_type, const AttnArgs &a, int64_t pairs, void *stream)
{
    const int slots = attn_slots(a.c.hd);
    void (*k)(AttnArgs) = nullptr;
#define QG_ATTN_T(T, DD) \
    a.side > 1 ? k_attn<T, DD, FORM, true> : k_attn<T, DD, FORM, false>
#define QG_ATTN_D(DD) k = kv_type == KV_F16 ? QG_ATTN_T(KV_F16, DD) : QG_ATTN_T(KV_BF16, DD)
    switch (a.c.hd) {
    case 64: QG_ATTN_D(64); break;
    case 96: QG_ATTN_D(96); break;
    case 128: QG_ATTN_D(128); break;
    case 192: QG_ATTN_D(192); break;
    default: QG_ATTN_D(256); break;
    }
#undef QG_ATTN_D
#undef QG_ATTN_T
    // as many pairs as slots: those that are much longer than the rest are split all the same
    const int64_t table = (int64_t)a.c.max_pages << a.c.ps_log2;
    const int64_t grid = pairs < slots ? slots : table > AttnCols::SOLO << AttnCols::UNIT_LOG2 ? pairs + slots : pairs;
    hipLaunchKernelGGL(k, dim3((unsigned)grid), dim3(256), 0, static_cast<hipStream_t>(stream), a);
    return (int)hipGetLastError();
}

int launch_attn(int kv_type, const AttnArgs &a, void *stream)
{
    AttnArgs b = a;
    b.side = (a.group + 15) / 16;
    return launch_k_attn<ONE>(kv_type, b, (int64_t)a.c.n_seq * a.c.nkv * b.side, stream);
}

int launch_attn_rows(int kv_type, const AttnArgs &a, void *stream)
{
    AttnArgs b = a;
    b.side = (int)((a.c.n_rows * a.group + 16 * a.c.n_seq - 1) / (16 * a.c.n_seq));   // on average
    return launch_k_attn<MANY>(kv_type, b, a.c.nkv * (a.c.n_rows * a.group / 16 + a.c.n_seq), stream);
}

}  // namespace qg
