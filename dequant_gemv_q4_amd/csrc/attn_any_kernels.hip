// attn_any_kernels.hip -- attention of one query row and head a workgroup, over pages of any type, its
// positions in tiles of 256: the plain form of the attentions over 8-bit pages and of shared prefixes.
#include <hip/hip_runtime.h>

#include "attn_common.h"

namespace qg {

template <int T>
__device__ __forceinline__ float value_at(const uint16_t *pages, int64_t block, int64_t at, int64_t scale_at)
{
    if constexpr (kv_bytes(T)) {
        const uint8_t *p = reinterpret_cast<const uint8_t *>(pages) + block;
        const float d = *reinterpret_cast<const float *>(p + scale_at);
        if constexpr (T == KV_I8)
            return d * (float)(int8_t)p[at];
        else
            return d * __builtin_amdgcn_cvt_f32_fp8(p[at], 0);
    } else {
        return low_of<T>(pages[block + at]);
    }
}

template <int T>
__global__ __launch_bounds__(256) void k_attn_any(AttnArgs a)
{
    __shared__ float s_q[256], s_p[256], s_w[4];
    __shared__ int s_page[256];
    const KvArgs &c = a.c;
    const int tid = threadIdx.x, head = blockIdx.y, h = head / a.group, ps = 1 << c.ps_log2;
    const int64_t row = blockIdx.x;
    int b = (int)row, len, first = b, shared = 0;
    if (c.q_start) {
        for (b = -1; b + 1 < c.n_seq && c.q_start[b + 1] <= row; ++b)
            ;
        if (b < 0 || row >= c.q_start[b + 1])
            return;
        first = b;
        len = c.kv_len[b] - (c.q_start[b + 1] - (int)row) + 1;
    } else {
        len = c.kv_len[b];
    }
    const int64_t cap = (int64_t)c.max_pages << c.ps_log2;
    if (len > cap) {
        atomicOr(c.err, 1u);
        len = (int)cap;
    }
    if (a.group_start)
        for (int g = 0; g < a.n_group; ++g) {
            const int f = max(a.group_start[g], 0);
            if (b >= f && b < a.group_start[g + 1]) {
                first = f;
                shared = min(a.shared_len[b], a.shared_len[f]);
                if (a.shared_len[b] > a.shared_len[f])
                    atomicOr(c.err, 1u);
            }
        }
    float o = 0.f, l = 0.f, m = -INFINITY;
    if (tid < c.hd)
        s_q[tid] = a.q[row * a.q_stride + (int64_t)head * c.hd + tid];
    for (int t0 = 0; t0 < len; t0 += 256) {
        __syncthreads();
        const int t = t0 + tid;
        int page = -1;
        float s = -INFINITY;
        if (t < len) {
            const int own = a.group_start && t >= shared && b != first && t < a.shared_len[b] ? -1 : 0;
            page = own < 0 ? -2 : c.table[(int64_t)(t < shared ? first : b) * c.max_pages + (t >> c.ps_log2)];
            if (page >= c.n_pages || page == -1 || page < -2) {
                atomicOr(c.err, 1u);
                page = -1;
            }
        }
        if (page >= 0) {
            const int64_t at = (int64_t)page * c.page_stride + (int64_t)h * c.block;
            const int slot = t & (ps - 1);
            s = 0.f;
            for (int d = 0; d < c.hd; ++d)
                s = fmaf(s_q[d], value_at<T>(c.k, at, slot * c.hd + d, (int64_t)c.hd * ps + 4 * slot), s);
            s *= a.scale * LOG2E;
        }
        s_page[tid] = page;
        float top = s;
#pragma unroll
        for (int x = 1; x < 64; x *= 2)
            top = fmaxf(top, __shfl_xor(top, x, 64));
        if (tid % 64 == 0)
            s_w[tid / 64] = top;
        __syncthreads();
        const float to = fmaxf(m, fmaxf(fmaxf(s_w[0], s_w[1]), fmaxf(s_w[2], s_w[3])));
        const float from = to == -INFINITY ? 0.f : to;
        s_p[tid] = page >= 0 ? __builtin_amdgcn_exp2f(s - from - 24.f) : 0.f;      // sums of values up to the type's end
        const float f = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - from);
        m = to;
        __syncthreads();
        o *= f;
        l *= f;
        for (int e = 0; e < 256 && t0 + e < len; ++e) {
            const int pg = s_page[e];
            if (pg < 0)
                continue;
            l += s_p[e];
            if (tid < c.hd) {
                const int slot = (t0 + e) & (ps - 1);
                o = fmaf(s_p[e], value_at<T>(c.v, (int64_t)pg * c.page_stride + (int64_t)h * c.block, tid * ps + slot,
                                             (int64_t)c.hd * ps + 4 * slot), o);
            }
        }
    }
    if (tid < c.hd)
        a.o[(row * a.nq + head) * c.hd + tid] = o * inverse_sum(l);
}

int launch_attn_any(int kv_type, const AttnArgs &a, void *stream)
{
    auto k = kv_type == KV_I8 ? k_attn_any<KV_I8> : kv_type == KV_F8 ? k_attn_any<KV_F8>
             : kv_type == KV_F16 ? k_attn_any<KV_F16> : k_attn_any<KV_BF16>;
    hipLaunchKernelGGL(k, dim3((unsigned)a.c.n_rows, (unsigned)a.nq), dim3(256), 0, static_cast<hipStream_t>(stream), a);
    return (int)hipGetLastError();
}

}  // namespace qg
