// attn_prompt_kernels.hip -- causal attention of packed rows.
#include <hip/hip_runtime.h>

#include "attn_common.h"

namespace qg {

// Round to nearest-even, as the conversion instructions do.
template <int T>
__device__ __forceinline__ uint16_t kv_round(float v)
{
    if constexpr (T == KV_F16)
        return __builtin_bit_cast(uint16_t, (_Float16)v);
    else
        return __builtin_bit_cast(uint16_t, (__bf16)v);
}
template <int T>
__device__ __forceinline__ float kv_float(uint16_t b)
{
    if constexpr (T == KV_F16)
        return (float)__builtin_bit_cast(_Float16, b);
    else
        return __builtin_bit_cast(float, (uint32_t)b << 16);
}

// Sequence of row r: the last b whose q_start is <= r and whose end is behind r, or -1.
__device__ __forceinline__ int seq_of_row(const KvArgs &c, int64_t r, int64_t &start, int64_t &end)
{
    if (!c.q_start) {
        start = r;
        end = r + 1;
        return (int)r;
    }
    for (int b = 0; b < c.n_seq; ++b) {
        start = c.q_start[b];
        end = c.q_start[b + 1];
        if (r >= start && r < end)
            return b;
    }
    return -1;
}

// Element offset of position t's page, or -1 (sticky flag set) if it has no valid one.
__device__ __forceinline__ int64_t page_at(const KvArgs &c, int b, int64_t t)
{
    const int64_t i = t >> c.ps_log2;
    const int page = i < c.max_pages ? c.table[(int64_t)b * c.max_pages + i] : -1;
    if (page < 0 || page >= c.n_pages) {
        atomicOr(c.err, 1u);
        return -1;
    }
    return page * c.page_stride;
}

// One workgroup per (row, query head): strips of 256 positions, a thread's score each, running
// maximum and sum, then each channel's weighted sum.
template <int T>
__global__ __launch_bounds__(256) void k_attn_plain(AttnArgs a)
{
    const KvArgs &c = a.c;
    __shared__ float sq[256], sp[256], red[4];
    __shared__ int64_t soff[256];
    const int64_t r = blockIdx.x;
    const int h = blockIdx.y, tid = threadIdx.x, hkv = h / a.group;
    int64_t start, end;
    const int b = seq_of_row(c, r, start, end);
    if (b < 0)
        return;
    const int64_t last = c.kv_len[b] - (end - r);       // the row's position
    for (int d = tid; d < c.hd; d += 256)
        sq[d] = a.q[r * a.q_stride + (int64_t)h * c.hd + d] * a.scale;
    float m = -INFINITY, l = 0.f, o = 0.f;
    __syncthreads();
    for (int64_t t0 = 0; t0 <= last && (t0 >> c.ps_log2) < c.max_pages; t0 += 256) {
        const int64_t t = t0 + tid;
        float s = -INFINITY;
        int64_t off = -1;
        if (t <= last)
            off = page_at(c, b, t);
        if (off >= 0) {
            off += ((int64_t)hkv * c.hd << c.ps_log2);
            const int slot = (int)(t & ((1 << c.ps_log2) - 1));
            s = 0.f;
            for (int d = 0; d < c.hd; ++d)
                s = fmaf(sq[d], kv_float<T>(c.k[off + (int64_t)slot * c.hd + d]), s);
            off += slot;
        }
        float mx = s;
        for (int x = 32; x; x >>= 1)
            mx = fmaxf(mx, __shfl_xor(mx, x));
        if ((tid & 63) == 0)
            red[tid >> 6] = mx;
        __syncthreads();
        mx = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
        const float mn = fmaxf(m, mx);
        const float p = off >= 0 ? expf(s - mn) : 0.f;
        const float f = m == -INFINITY ? 0.f : expf(m - mn);
        sp[tid] = p;
        soff[tid] = off;
        __syncthreads();
        o *= f;
        l *= f;
        m = mn;
        for (int j = 0; j < 256; ++j) {
            l += sp[j];
            if (soff[j] >= 0 && tid < c.hd)
                o = fmaf(sp[j], kv_float<T>(c.v[soff[j] + ((int64_t)tid << c.ps_log2)]), o);
        }
        __syncthreads();
    }
    if (tid < c.hd)
        a.o[r * a.nq * c.hd + (int64_t)h * c.hd + tid] = m == -INFINITY ? 0.f : o / l;
}

static int launch_plain(int kv_type, const AttnArgs &a, void *stream)
{
    hipStream_t s = static_cast<hipStream_t>(stream);
    const dim3 grid((unsigned)a.c.n_rows, (unsigned)a.nq);
    if (kv_type == KV_F16)
        hipLaunchKernelGGL(k_attn_plain<KV_F16>, grid, dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL(k_attn_plain<KV_BF16>, grid, dim3(256), 0, s, a);
    return (int)hipGetLastError();
}

int launch_attn_prompt(int kv_type, const AttnArgs &a, void *stream) { return launch_plain(kv_type, a, stream); }

}  // namespace qg
