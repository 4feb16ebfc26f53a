// abi_attn.cpp -- the C ABI of the attention side: the paged key-value cache, what writes it,
// attention over it and expert routing.  As in abi.cpp, every argument is validated on the host before anything is
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

// Workspace: the sticky flag (256 bytes) and the arrival counters (of a split joined in its launch, of one behind
// a shared prefix, and of a row's halves), at the same place for every operation (the counters are 0 between calls
// and must stay so when operations share a workspace), then what an operation writes before it reads.
static constexpr int64_t WS_COUNT = 256, WS_TAIL = WS_COUNT + ATTN_MAX_SLOTS * 4;
static constexpr int64_t WS_MEET = WS_TAIL + ATTN_MAX_SLOTS * 4, WS_PART = WS_MEET + MEET_MOST * 4;
// qgemv_attn_prompt's part of it begins with its pair count and its split tiles (32 bytes each).
static constexpr int64_t WS_SPLITS = 256 + PROMPT_SPLITS * 32;

static int64_t rounded_up(int64_t bytes) { return (bytes + 255) / 256 * 256; }

// Partial results of a split over 16-column and over 128-column tiles.
static int64_t parts_16(int nq, int nkv, int hd)
{
    const int group = nq / nkv;
    return rounded_up(attn_slots(hd) * attn_part_floats(group < 16 ? group : 16, hd) * 4);
}
static int64_t parts_128(int hd) { return WS_SPLITS + (int64_t)prompt_slots(hd) * 128 * (hd + 2) * 4; }

// qgemv_attn_shared: exponents and sums of both halves, and their means where they meet in one launch.
static int64_t stats_bytes(int n_seq, int nq) { return rounded_up((int64_t)n_seq * nq * 2 * 8); }
static int64_t means_bytes(int n_seq, int nq, int hd)
{
    const int64_t rows = (int64_t)n_seq * nq;
    return rows > MEET_MOST ? 0 : rounded_up(rows * hd * 2 * 4);
}

static int64_t ws_bytes_of(int op, int n_seq, int nq, int nkv, int hd)
{
    switch (op) {
    case QG_OP_ATTN: return WS_PART + parts_16(nq, nkv, hd);
    case QG_OP_ATTN_PROMPT: return WS_PART + parts_128(hd);
    case QG_OP_ATTN_SHARED:
        return WS_PART + stats_bytes(n_seq, nq) + means_bytes(n_seq, nq, hd) + parts_16(nq, nkv, hd) + parts_128(hd);
    default: return WS_TAIL;
    }
}

struct Span {
    const void *p;
    int64_t n;
};

// Checks of the cache and the metadata shared by the five calls that take a cache; fills c and the
// byte span of either page array.
static int check_cache(int kv_type, const void *k_pages, const void *v_pages, int64_t n_pages,
                       int page_size, int64_t page_stride, int nq, int nkv, int hd,
                       const int32_t *table, int max_pages, const int32_t *q_start,
                       const int32_t *kv_len, int n_seq, int64_t n_rows, KvArgs *c, int64_t *span)
{
    if (kv_type != QG_F16 && kv_type != QG_BF16 && kv_type != QG_I8 && kv_type != QG_F8)
        return QG_ERR_FORMAT;
    const bool bytes = kv_bytes(kv_type);
    if (!k_pages || !v_pages || !table || !kv_len)
        return QG_ERR_NULL;
    int lg = 4;
    while (lg < 8 && (1 << lg) != page_size)
        ++lg;
    if ((1 << lg) != page_size || !heads_ok(nq, nkv, hd) || n_seq < 1 || n_seq > QG_ATTN_MAX_SEQ ||
        n_rows < 1 || n_rows > QG_GEMM_MAX_M || max_pages < 1 ||
        (int64_t)max_pages * page_size > (1 << 24) || n_pages < 1 || n_pages > (1 << 28) ||
        page_stride % (bytes ? 16 : 8) || page_stride >= ((int64_t)1 << 32) ||
        (int64_t)nkv * page_size * hd > (1 << 28))
        return QG_ERR_SHAPE;
    const int64_t block = (int64_t)page_size * (bytes ? hd + 4 : hd);
    if (page_stride < nkv * block)
        return QG_ERR_SHAPE;
    if (!al(k_pages, 16) || !al(v_pages, 16) || !al(table, 4) || !al(kv_len, 4) ||
        (q_start && !al(q_start, 4)))
        return QG_ERR_ALIGN;
    memset(c, 0, sizeof(*c));
    c->k = static_cast<uint16_t *>(const_cast<void *>(k_pages));
    c->v = static_cast<uint16_t *>(const_cast<void *>(v_pages));
    c->page_stride = page_stride;
    c->block = block;
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
    *span = ((n_pages - 1) * page_stride + nkv * block) * (bytes ? 1 : 2);
    return QG_OK;
}

static bool hits(const void *p, int64_t n, const Span *s, int count)
{
    for (int i = 0; i < count; ++i)
        if (s[i].p && overlap(p, n, s[i].p, s[i].n))
            return true;
    return false;
}

// Checks of the workspace and of the page arrays as outputs, shared by the calls that write the cache.
static int check_written(int kv_type, const KvArgs &c, int64_t span, const Span *in, int n_in, void *ws,
                         size_t ws_bytes, int op)
{
    if (!ws)
        return QG_ERR_WORKSPACE;
    if (!al(ws, 256))
        return QG_ERR_ALIGN;
    if ((int64_t)ws_bytes < ws_bytes_of(op, c.n_seq, c.nkv, c.nkv, c.hd))
        return QG_ERR_WORKSPACE;
    const Span pages[] = {{c.k, span}, {c.v, span}};
    if (hits(c.k, span, in, n_in) || hits(c.v, span, in, n_in) || hits(ws, (int64_t)ws_bytes, in, n_in) ||
        hits(ws, (int64_t)ws_bytes, pages, 2))
        return QG_ERR_ALIAS;
    // one pool may interleave K and V, but their blocks within a page may not overlap
    const int64_t size = kv_bytes(kv_type) ? 1 : 2, block = c.nkv * c.block * size, step = c.page_stride * size;
    const int64_t apart = (int64_t)((uintptr_t)c.v - (uintptr_t)c.k), rem = (apart % step + step) % step;
    if (overlap(c.k, span, c.v, span) && (rem < block || step - rem < block))
        return QG_ERR_ALIAS;
    return QG_OK;
}

// The groups of qgemv_attn_shared.
struct Groups {
    const int32_t *start, *shared;
    int n;
};

// op: QG_OP_ATTN, QG_OP_ATTN_PROMPT or QG_OP_ATTN_SHARED.
static int run_attn(int op, int kv_type, const void *k_pages, const void *v_pages,
                    int64_t n_pages, int page_size, int64_t page_stride, int nkv, int hd,
                    const int32_t *table, int max_pages, const int32_t *q_start,
                    const int32_t *kv_len, int n_seq, const Groups &groups, const float *q,
                    int64_t q_stride, int64_t n_rows, int nq, float scale, float *o, void *ws,
                    size_t ws_bytes, void *stream)
{
    const bool prompt = op == QG_OP_ATTN_PROMPT, shared = op == QG_OP_ATTN_SHARED;
    AttnArgs a;
    memset(&a, 0, sizeof(a));
    int64_t span = 0;
    const int st = check_cache(kv_type, k_pages, v_pages, n_pages, page_size, page_stride, nq, nkv,
                               hd, table, max_pages, q_start, kv_len, n_seq, n_rows, &a.c, &span);
    if (st != QG_OK)
        return st;
    if (!q || !o || (prompt && !q_start) || (shared && (!groups.start || !groups.shared)))
        return QG_ERR_NULL;
    const int64_t width = (int64_t)nq * hd;
    if (q_stride < width || q_stride > ((int64_t)1 << 31) || n_rows * nq > (1 << 30) ||
        !isfinite(scale) || (shared && (groups.n < 1 || groups.n > n_seq)))
        return QG_ERR_SHAPE;
    if (prompt && plan_prompt(n_rows, n_seq, nkv, nq / nkv, hd, 0).pairs > 0x7fffffffLL)
        return QG_ERR_SHAPE;
    if (!al(q, 16) || !al(o, 16) || q_stride % 4 || !al(groups.start, 4) || !al(groups.shared, 4))
        return QG_ERR_ALIGN;
    if (!ws)
        return QG_ERR_WORKSPACE;
    if (!al(ws, 256))
        return QG_ERR_ALIGN;
    if ((int64_t)ws_bytes < ws_bytes_of(op, n_seq, nq, nkv, hd))
        return QG_ERR_WORKSPACE;
    const Span in[] = {{q, ((n_rows - 1) * q_stride + width) * 4},
                       {k_pages, span},
                       {v_pages, span},
                       {table, (int64_t)n_seq * max_pages * 4},
                       {kv_len, (int64_t)n_seq * 4},
                       {q_start, (int64_t)(n_seq + 1) * 4},
                       {groups.start, (int64_t)(groups.n + 1) * 4},
                       {groups.shared, (int64_t)n_seq * 4}};
    if (hits(o, n_rows * width * 4, in, 8) || hits(ws, (int64_t)ws_bytes, in, 8) ||
        overlap(o, n_rows * width * 4, ws, (int64_t)ws_bytes))
        return QG_ERR_ALIAS;
    a.c.err = static_cast<unsigned int *>(ws);
    a.count = reinterpret_cast<unsigned int *>(static_cast<uint8_t *>(ws) + WS_COUNT);
    uint8_t *const w = static_cast<uint8_t *>(ws), *part = w + WS_PART;
    if (shared) {
        a.meet = reinterpret_cast<unsigned int *>(w + WS_MEET);
        a.tail_count = reinterpret_cast<unsigned int *>(w + WS_TAIL);
        a.stats = reinterpret_cast<float *>(part);
        part += stats_bytes(n_seq, nq);
        a.means = reinterpret_cast<float *>(part);
        part += means_bytes(n_seq, nq, hd);
        a.tail_part = reinterpret_cast<float *>(part);
        part += parts_16(nq, nkv, hd);
    }
    a.pairs = reinterpret_cast<int *>(part);
    a.splits = reinterpret_cast<PromptSplit *>(part + 256);
    a.part = reinterpret_cast<float *>(prompt || shared ? part + WS_SPLITS : part);
    a.rows_in_all = n_seq;
    a.q = q;
    a.q_stride = q_stride;
    a.o = o;
    a.nq = nq;
    a.group = nq / nkv;
    a.scale = scale;
    a.group_start = groups.start;
    a.shared_len = groups.shared;
    a.n_group = groups.n;
    const bool bytes = kv_bytes(kv_type);
    return launch_status(shared   ? launch_attn_shared(kv_type, a, stream)
                         : prompt ? launch_attn_prompt(kv_type, a, stream)
                         : bytes  ? launch_attn8(kv_type, a, stream)
                                  : launch_attn(kv_type, a, stream));
}

extern "C" {

int64_t qgemv_attn_workspace_bytes(int op, int n_seq, int n_q_heads, int n_kv_heads, int head_dim)
{
    if (op < QG_OP_KV_APPEND || op > QG_OP_ATTN_SHARED || n_seq < 1 ||
        n_seq > QG_ATTN_MAX_SEQ || !heads_ok(n_q_heads, n_kv_heads, head_dim))
        return -1;
    return ws_bytes_of(op, n_seq, n_q_heads, n_kv_heads, head_dim);
}

int qgemv_kv_append(int kv_type, void *k_pages, void *v_pages, int64_t n_pages, int page_size,
                    int64_t page_stride, int n_kv_heads, int head_dim, const int32_t *table,
                    int max_pages, const int32_t *q_start, const int32_t *kv_len, int n_seq,
                    const float *k, const float *v, int64_t kv_stride, int64_t n_rows, void *ws,
                    size_t ws_bytes, void *stream)
{
    AppendArgs a;
    int64_t span = 0;
    int st = check_cache(kv_type, k_pages, v_pages, n_pages, page_size, page_stride, n_kv_heads,
                         n_kv_heads, head_dim, table, max_pages, q_start, kv_len, n_seq, n_rows, &a.c,
                         &span);
    if (st != QG_OK)
        return st;
    if (!k || !v)
        return QG_ERR_NULL;
    const int64_t width = (int64_t)n_kv_heads * head_dim;
    if (kv_stride < width || kv_stride > ((int64_t)1 << 31) || (!q_start && n_rows != n_seq))
        return QG_ERR_SHAPE;
    if (!al(k, 16) || !al(v, 16) || kv_stride % 4)
        return QG_ERR_ALIGN;
    const int64_t rows = ((n_rows - 1) * kv_stride + width) * 4;
    const Span in[] = {{k, rows},
                       {v, rows},
                       {table, (int64_t)n_seq * max_pages * 4},
                       {kv_len, (int64_t)n_seq * 4},
                       {q_start, (int64_t)(n_seq + 1) * 4}};
    st = check_written(kv_type, a.c, span, in, 5, ws, ws_bytes, QG_OP_KV_APPEND);
    if (st != QG_OK)
        return st;
    a.c.err = static_cast<unsigned int *>(ws);
    a.ksrc = k;
    a.vsrc = v;
    a.stride = kv_stride;
    if (!kv_bytes(kv_type))
        return launch_status(launch_kv_append(kv_type, a, stream));
    QkvArgs b;
    memset(&b, 0, sizeof(b));
    b.c = a.c;
    b.k = k;
    b.v = v;
    b.stride = kv_stride;
    return launch_status(launch_qkv_append(kv_type, false, b, stream));
}

int qgemv_qkv_append(int kv_type, void *k_pages, void *v_pages, int64_t n_pages, int page_size,
                     int64_t page_stride, int n_kv_heads, int head_dim, const int32_t *table,
                     int max_pages, const int32_t *q_start, const int32_t *kv_len, int n_seq,
                     const float *qkv, int64_t qkv_stride, int64_t n_rows, int n_q_heads,
                     int rope_half, const float *q_gamma, const float *k_gamma, float eps,
                     const float *rope_cos, const float *rope_sin, int64_t rope_rows, float *q,
                     int64_t q_stride, void *ws, size_t ws_bytes, void *stream)
{
    QkvArgs a;
    memset(&a, 0, sizeof(a));
    int64_t span = 0;
    int st = check_cache(kv_type, k_pages, v_pages, n_pages, page_size, page_stride, n_q_heads,
                         n_kv_heads, head_dim, table, max_pages, q_start, kv_len, n_seq, n_rows, &a.c,
                         &span);
    if (st != QG_OK)
        return st;
    if (!qkv || !q || (rope_half > 0 && (!rope_cos || !rope_sin)))
        return QG_ERR_NULL;
    const int64_t q_width = (int64_t)n_q_heads * head_dim;
    const int64_t width = q_width + 2 * (int64_t)n_kv_heads * head_dim, most = (int64_t)1 << 31;
    if (qkv_stride < width || qkv_stride > most || q_stride < q_width || q_stride > most ||
        (!q_start && n_rows != n_seq) || n_rows * n_q_heads > (1 << 30) || rope_half < 0 ||
        rope_half > head_dim / 2 || !isfinite(eps) || eps < 0.f ||
        (rope_half > 0 && (rope_rows < 1 || rope_rows > (1 << 24))))
        return QG_ERR_SHAPE;
    if (!rope_half)
        rope_cos = rope_sin = nullptr;
    if (!al(qkv, 16) || !al(q, 16) || qkv_stride % 4 || q_stride % 4 || !al(q_gamma, 16) ||
        !al(k_gamma, 16) || !al(rope_cos, 16) || !al(rope_sin, 16))
        return QG_ERR_ALIGN;
    const bool in_place = q == qkv && q_stride == qkv_stride;
    const int64_t rows = ((n_rows - 1) * qkv_stride + width) * 4, turns = rope_rows * rope_half * 4;
    const int64_t q_span = ((n_rows - 1) * q_stride + q_width) * 4, head = (int64_t)head_dim * 4;
    const Span in[] = {{qkv, rows},
                       {table, (int64_t)n_seq * max_pages * 4},
                       {kv_len, (int64_t)n_seq * 4},
                       {q_start, (int64_t)(n_seq + 1) * 4},
                       {q_gamma, head},
                       {k_gamma, head},
                       {rope_cos, turns},
                       {rope_sin, turns},
                       {q, q_span}};
    st = check_written(kv_type, a.c, span, in, 9, ws, ws_bytes, QG_OP_QKV_APPEND);
    if (st != QG_OK)
        return st;
    if (hits(q, q_span, in + 1, 7) || (!in_place && overlap(q, q_span, qkv, rows)))
        return QG_ERR_ALIAS;
    a.c.err = static_cast<unsigned int *>(ws);
    a.q = qkv;
    a.k = qkv + q_width;
    a.v = a.k + (int64_t)n_kv_heads * head_dim;
    a.stride = qkv_stride;
    a.qo = q;
    a.qo_stride = q_stride;
    a.q_gamma = q_gamma;
    a.k_gamma = k_gamma;
    a.cos = rope_cos;
    a.sin = rope_sin;
    a.rope_rows = rope_half ? rope_rows : 0;
    a.nq = n_q_heads;
    a.half = rope_half;
    a.eps = eps;
    return launch_status(launch_qkv_append(kv_type, true, a, stream));
}

int qgemv_attn(int kv_type, const void *k_pages, const void *v_pages, int64_t n_pages,
               int page_size, int64_t page_stride, int n_kv_heads, int head_dim,
               const int32_t *table, int max_pages, const int32_t *kv_len, int n_seq,
               const float *q, int64_t q_stride, int n_q_heads, float scale, float *o, void *ws,
               size_t ws_bytes, void *stream)
{
    return run_attn(QG_OP_ATTN, kv_type, k_pages, v_pages, n_pages, page_size, page_stride, n_kv_heads,
                    head_dim, table, max_pages, nullptr, kv_len, n_seq, Groups{}, q, q_stride,
                    n_seq, n_q_heads, scale, o, ws, ws_bytes, stream);
}

int qgemv_attn_prompt(int kv_type, const void *k_pages, const void *v_pages, int64_t n_pages,
                      int page_size, int64_t page_stride, int n_kv_heads, int head_dim,
                      const int32_t *table, int max_pages, const int32_t *q_start,
                      const int32_t *kv_len, int n_seq, const float *q, int64_t q_stride,
                      int64_t n_rows, int n_q_heads, float scale, float *o, void *ws,
                      size_t ws_bytes, void *stream)
{
    return run_attn(QG_OP_ATTN_PROMPT, kv_type, k_pages, v_pages, n_pages, page_size, page_stride, n_kv_heads,
                    head_dim, table, max_pages, q_start, kv_len, n_seq, Groups{}, q, q_stride,
                    n_rows, n_q_heads, scale, o, ws, ws_bytes, stream);
}

int qgemv_attn_shared(int kv_type, const void *k_pages, const void *v_pages, int64_t n_pages,
                      int page_size, int64_t page_stride, int n_kv_heads, int head_dim,
                      const int32_t *table, int max_pages, const int32_t *kv_len, int n_seq,
                      const int32_t *group_start, const int32_t *shared_len, int n_group,
                      const float *q, int64_t q_stride, int n_q_heads, float scale, float *o, void *ws,
                      size_t ws_bytes, void *stream)
{
    return run_attn(QG_OP_ATTN_SHARED, kv_type, k_pages, v_pages, n_pages, page_size, page_stride,
                    n_kv_heads, head_dim, table, max_pages, nullptr, kv_len, n_seq,
                    Groups{group_start, shared_len, n_group}, q, q_stride, n_seq, n_q_heads, scale, o,
                    ws, ws_bytes, stream);
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
