// abi_attn.cpp -- the C ABI of the attention side: the paged key-value cache, attention over it
// and expert routing.  As in abi.cpp, every argument is validated on the host before anything is
// launched; what only the device knows (lengths, page tables) the kernels check themselves.
#include <hip/hip_runtime.h>

#include <math.h>
#include <string.h>

#include "../../include/qgemv.h"
#include "attn_internal.h"

using namespace qg;

static bool al(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

static bool overlap(const void *a, int64_t na, const void *b, int64_t nb)
{
    const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
    return a0 < b0 + (uintptr_t)nb && b0 < a0 + (uintptr_t)na;
}

static int launch_status(int herr) { return herr == 0 ? QG_OK : QG_ERR_LAUNCH; }

static bool head_dim_ok(int hd) { return hd == 64 || hd == 96 || hd == 128 || hd == 192 || hd == 256; }

static bool heads_ok(int nq, int nkv, int hd)
{
    return nkv >= 1 && nq >= nkv && nq % nkv == 0 && head_dim_ok(hd) && nq <= 4096;
}

// Workspace: the sticky flag (256 bytes) and the arrival counters of a split joined in its launch, at the same
// place for every operation (the counters are 0 between calls and must stay so when operations share
// a workspace), then the partial results of a split.
static constexpr int64_t WS_COUNT = 256, WS_PART = WS_COUNT + ATTN_MAX_SLOTS * 4;
// qgemv_attn_prompt's part of it begins with its pair count and its split tiles (32 bytes each).
static constexpr int64_t WS_SPLITS = 256 + PROMPT_SPLITS * 32;

static int64_t ws_bytes_of(int op, int nq, int nkv, int hd)
{
    const int group = nq / nkv;
    if (op == QG_OP_ATTN)
        return WS_PART + (attn_slots(hd) * attn_part_floats(group < 16 ? group : 16, hd) * 4 + 255) / 256 * 256;
    if (op == QG_OP_ATTN_PROMPT)
        return WS_PART + WS_SPLITS + (int64_t)prompt_slots(hd) * 128 * (hd + 2) * 4;   // 128 columns a tile
    return WS_PART;
}

struct Span {
    const void *p;
    int64_t n;
};

// Checks of the cache and the metadata shared by the three calls; fills c and the byte span of
// either page array.
static int check_cache(int kv_type, const void *k_pages, const void *v_pages, int64_t n_pages,
                       int page_size, int64_t page_stride, int nq, int nkv, int hd,
                       const int32_t *table, int max_pages, const int32_t *q_start,
                       const int32_t *kv_len, int n_seq, int64_t n_rows, KvArgs *c, int64_t *span)
{
    if (kv_type != QG_F16 && kv_type != QG_BF16)
        return QG_ERR_FORMAT;
    if (!k_pages || !v_pages || !table || !kv_len)
        return QG_ERR_NULL;
    int lg = 4;
    while (lg < 8 && (1 << lg) != page_size)
        ++lg;
    if ((1 << lg) != page_size || !heads_ok(nq, nkv, hd) || n_seq < 1 || n_seq > QG_ATTN_MAX_SEQ ||
        n_rows < 1 || n_rows > QG_GEMM_MAX_M || max_pages < 1 ||
        (int64_t)max_pages * page_size > (1 << 24) || n_pages < 1 || n_pages > (1 << 28) ||
        page_stride % 8 || page_stride < (int64_t)nkv * page_size * hd ||
        page_stride >= ((int64_t)1 << 32) || (int64_t)nkv * page_size * hd > (1 << 28))
        return QG_ERR_SHAPE;
    if (!al(k_pages, 16) || !al(v_pages, 16) || !al(table, 4) || !al(kv_len, 4) ||
        (q_start && !al(q_start, 4)))
        return QG_ERR_ALIGN;
    memset(c, 0, sizeof(*c));
    c->k = static_cast<uint16_t *>(const_cast<void *>(k_pages));
    c->v = static_cast<uint16_t *>(const_cast<void *>(v_pages));
    c->page_stride = page_stride;
    c->n_pages = n_pages;
    c->table = table;
    c->q_start = q_start;
    c->kv_len = kv_len;
    c->max_pages = max_pages;
    c->n_seq = n_seq;
    c->ps_log2 = lg;
    c->nkv = nkv;
    c->hd = hd;
    c->n_rows = n_rows;
    *span = ((n_pages - 1) * page_stride + (int64_t)nkv * page_size * hd) * 2;
    return QG_OK;
}

static bool hits(const void *p, int64_t n, const Span *s, int count)
{
    for (int i = 0; i < count; ++i)
        if (s[i].p && overlap(p, n, s[i].p, s[i].n))
            return true;
    return false;
}

static int run_attn(bool prompt, int kv_type, const void *k_pages, const void *v_pages,
                    int64_t n_pages, int page_size, int64_t page_stride, int nkv, int hd,
                    const int32_t *table, int max_pages, const int32_t *q_start,
                    const int32_t *kv_len, int n_seq, const float *q, int64_t q_stride,
                    int64_t n_rows, int nq, float scale, float *o, void *ws, size_t ws_bytes,
                    void *stream)
{
    AttnArgs a;
    memset(&a, 0, sizeof(a));
    int64_t span = 0;
    const int st = check_cache(kv_type, k_pages, v_pages, n_pages, page_size, page_stride, nq, nkv,
                               hd, table, max_pages, q_start, kv_len, n_seq, n_rows, &a.c, &span);
    if (st != QG_OK)
        return st;
    if (!q || !o || (prompt && !q_start))
        return QG_ERR_NULL;
    const int64_t width = (int64_t)nq * hd;
    if (q_stride < width || q_stride > ((int64_t)1 << 31) || n_rows * nq > (1 << 30) ||
        !isfinite(scale))
        return QG_ERR_SHAPE;
    if (prompt && plan_prompt(n_rows, n_seq, nkv, nq / nkv, hd, 0).pairs > 0x7fffffffLL)
        return QG_ERR_SHAPE;
    if (!al(q, 16) || !al(o, 16) || q_stride % 4)
        return QG_ERR_ALIGN;
    if (!ws)
        return QG_ERR_WORKSPACE;
    if (!al(ws, 256))
        return QG_ERR_ALIGN;
    if ((int64_t)ws_bytes < ws_bytes_of(prompt ? QG_OP_ATTN_PROMPT : QG_OP_ATTN, nq, nkv, hd))
        return QG_ERR_WORKSPACE;
    const Span in[] = {{q, ((n_rows - 1) * q_stride + width) * 4},
                       {k_pages, span},
                       {v_pages, span},
                       {table, (int64_t)n_seq * max_pages * 4},
                       {kv_len, (int64_t)n_seq * 4},
                       {q_start, (int64_t)(n_seq + 1) * 4}};
    if (hits(o, n_rows * width * 4, in, 6) || hits(ws, (int64_t)ws_bytes, in, 6) ||
        overlap(o, n_rows * width * 4, ws, (int64_t)ws_bytes))
        return QG_ERR_ALIAS;
    a.c.err = static_cast<unsigned int *>(ws);
    a.count = reinterpret_cast<unsigned int *>(static_cast<uint8_t *>(ws) + WS_COUNT);
    uint8_t *part = static_cast<uint8_t *>(ws) + WS_PART;
    a.pairs = reinterpret_cast<int *>(part);
    a.splits = reinterpret_cast<PromptSplit *>(part + 256);
    a.part = reinterpret_cast<float *>(prompt ? part + WS_SPLITS : part);
    a.q = q;
    a.q_stride = q_stride;
    a.o = o;
    a.nq = nq;
    a.group = nq / nkv;
    a.scale = scale;
    return launch_status(prompt ? launch_attn_prompt(kv_type, a, stream)
                                : launch_attn(kv_type, a, stream));
}

extern "C" {

int64_t qgemv_attn_workspace_bytes(int op, int n_seq, int n_q_heads, int n_kv_heads, int head_dim)
{
    if ((op != QG_OP_KV_APPEND && op != QG_OP_ATTN && op != QG_OP_ATTN_PROMPT) || n_seq < 1 ||
        n_seq > QG_ATTN_MAX_SEQ || !heads_ok(n_q_heads, n_kv_heads, head_dim))
        return -1;
    return ws_bytes_of(op, n_q_heads, n_kv_heads, head_dim);
}

int qgemv_kv_append(int kv_type, void *k_pages, void *v_pages, int64_t n_pages, int page_size,
                    int64_t page_stride, int n_kv_heads, int head_dim, const int32_t *table,
                    int max_pages, const int32_t *q_start, const int32_t *kv_len, int n_seq,
                    const float *k, const float *v, int64_t kv_stride, int64_t n_rows, void *ws,
                    size_t ws_bytes, void *stream)
{
    AppendArgs a;
    int64_t span = 0;
    const int st = check_cache(kv_type, k_pages, v_pages, n_pages, page_size, page_stride,
                               n_kv_heads, n_kv_heads, head_dim, table, max_pages, q_start, kv_len,
                               n_seq, n_rows, &a.c, &span);
    if (st != QG_OK)
        return st;
    if (!k || !v)
        return QG_ERR_NULL;
    const int64_t width = (int64_t)n_kv_heads * head_dim;
    if (kv_stride < width || kv_stride > ((int64_t)1 << 31) || (!q_start && n_rows != n_seq))
        return QG_ERR_SHAPE;
    if (!al(k, 16) || !al(v, 16) || kv_stride % 4)
        return QG_ERR_ALIGN;
    if (!ws)
        return QG_ERR_WORKSPACE;
    if (!al(ws, 256))
        return QG_ERR_ALIGN;
    if ((int64_t)ws_bytes < ws_bytes_of(QG_OP_KV_APPEND, n_kv_heads, n_kv_heads, head_dim))
        return QG_ERR_WORKSPACE;
    const int64_t rows = ((n_rows - 1) * kv_stride + width) * 4;
    const Span in[] = {{k, rows},
                       {v, rows},
                       {table, (int64_t)n_seq * max_pages * 4},
                       {kv_len, (int64_t)n_seq * 4},
                       {q_start, (int64_t)(n_seq + 1) * 4}};
    const Span pages[] = {{k_pages, span}, {v_pages, span}};
    if (hits(k_pages, span, in, 5) || hits(v_pages, span, in, 5) ||
        hits(ws, (int64_t)ws_bytes, in, 5) || hits(ws, (int64_t)ws_bytes, pages, 2))
        return QG_ERR_ALIAS;
    // one pool may interleave K and V, but their blocks within a page may not overlap
    const int64_t block = width * page_size * 2;
    const int64_t apart = (int64_t)((uintptr_t)v_pages - (uintptr_t)k_pages);
    const int64_t rem = ((apart % (page_stride * 2)) + page_stride * 2) % (page_stride * 2);
    if (overlap(k_pages, span, v_pages, span) && (rem < block || page_stride * 2 - rem < block))
        return QG_ERR_ALIAS;
    a.c.err = static_cast<unsigned int *>(ws);
    a.ksrc = k;
    a.vsrc = v;
    a.stride = kv_stride;
    return launch_status(launch_kv_append(kv_type, a, stream));
}

int qgemv_attn(int kv_type, const void *k_pages, const void *v_pages, int64_t n_pages,
               int page_size, int64_t page_stride, int n_kv_heads, int head_dim,
               const int32_t *table, int max_pages, const int32_t *kv_len, int n_seq,
               const float *q, int64_t q_stride, int n_q_heads, float scale, float *o, void *ws,
               size_t ws_bytes, void *stream)
{
    return run_attn(false, kv_type, k_pages, v_pages, n_pages, page_size, page_stride, n_kv_heads,
                    head_dim, table, max_pages, nullptr, kv_len, n_seq, q, q_stride, n_seq,
                    n_q_heads, scale, o, ws, ws_bytes, stream);
}

int qgemv_attn_prompt(int kv_type, const void *k_pages, const void *v_pages, int64_t n_pages,
                      int page_size, int64_t page_stride, int n_kv_heads, int head_dim,
                      const int32_t *table, int max_pages, const int32_t *q_start,
                      const int32_t *kv_len, int n_seq, const float *q, int64_t q_stride,
                      int64_t n_rows, int n_q_heads, float scale, float *o, void *ws,
                      size_t ws_bytes, void *stream)
{
    return run_attn(true, kv_type, k_pages, v_pages, n_pages, page_size, page_stride, n_kv_heads,
                    head_dim, table, max_pages, q_start, kv_len, n_seq, q, q_stride, n_rows,
                    n_q_heads, scale, o, ws, ws_bytes, stream);
}

int qgemv_attn_error(const void *ws, int *flag, void *stream)
{
    if (!ws || !flag)
        return QG_ERR_NULL;
    unsigned int v = 0;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (hipMemcpyAsync(&v, ws, 4, hipMemcpyDeviceToHost, s) != hipSuccess ||
        hipStreamSynchronize(s) != hipSuccess)
        return QG_ERR_LAUNCH;
    *flag = (int)v;
    if (v) {
        const unsigned int zero = 0;
        if (hipMemcpyAsync(const_cast<void *>(ws), &zero, 4, hipMemcpyHostToDevice, s) != hipSuccess ||
            hipStreamSynchronize(s) != hipSuccess)
            return QG_ERR_LAUNCH;
    }
    return QG_OK;
}

int qgemv_route(const float *logits, int64_t n_rows, int n_exp, int score, const float *bias,
                int n_group, int group_top, int topk_group, int topk, int renorm, float scale,
                int32_t *ids, float *wts, void *stream)
{
    if (!logits || !ids || !wts)
        return QG_ERR_NULL;
    if (n_rows < 1 || n_rows > QG_GEMM_MAX_M || n_exp < 1 || n_exp > QG_ROUTE_MAX_EXP ||
        (score != QG_SCORE_SOFTMAX && score != QG_SCORE_SIGMOID) || n_group < 1 ||
        n_group > n_exp || n_exp % n_group || group_top < 1 || group_top > 2 ||
        group_top > n_exp / n_group || topk_group < 1 || topk_group > n_group || topk < 1 ||
        topk > QG_MAX_TOPK || topk > topk_group * (n_exp / n_group) || !isfinite(scale))
        return QG_ERR_SHAPE;
    if (!al(logits, 4) || (bias && !al(bias, 4)) || !al(ids, 4) || !al(wts, 4))
        return QG_ERR_ALIGN;
    const int64_t out = n_rows * topk * 4;
    const Span in[] = {{logits, n_rows * n_exp * 4}, {bias, (int64_t)n_exp * 4}};
    if (hits(ids, out, in, 2) || hits(wts, out, in, 2) || overlap(ids, out, wts, out))
        return QG_ERR_ALIAS;
    RouteArgs a;
    memset(&a, 0, sizeof(a));
    a.z = logits;
    a.bias = bias;
    a.ids = ids;
    a.wts = wts;
    a.n_rows = n_rows;
    a.n_exp = n_exp;
    a.sigmoid = score == QG_SCORE_SIGMOID;
    a.n_group = n_group;
    a.group_top = group_top;
    a.topk_group = n_group > 1 ? topk_group : 1;
    a.topk = topk;
    a.renorm = renorm != 0;
    a.scale = scale;
    return launch_status(launch_route(a, stream));
}

}  // extern "C"
