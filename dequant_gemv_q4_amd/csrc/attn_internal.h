// attn_internal.h -- library-internal declarations of the attention side (paged key-value cache,
// attention, expert routing) shared by abi_attn.cpp and its kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace qg {

// Workgroup slots of the split over a cache's length (qgemv_attn): two per compute unit.
#define ATTN_SLOTS 512
// The same of qgemv_attn_prompt: tile splits, and with them partial results, of a call.
#define PROMPT_SLOTS 512

enum KvType { KV_F16 = 1, KV_BF16 = 30 };

// The paged cache and the step's metadata, as the public header describes them.
struct KvArgs {
    uint16_t *k, *v;            // page arrays (2-byte elements)
    int64_t page_stride;        // elements from page to page
    int64_t n_pages;
    const int32_t *table;       // [n_seq][max_pages]
    const int32_t *q_start;     // [n_seq + 1], or NULL: one row per sequence
    const int32_t *kv_len;      // [n_seq]
    unsigned int *err;          // workspace: sticky flag (bit 0: a position without a valid page)
    int max_pages, n_seq;
    int ps_log2;                // log2 of the page size
    int nkv, hd;
    int64_t n_rows;
};

struct AppendArgs {
    KvArgs c;
    const float *ksrc, *vsrc;   // row 0 of the new K and V
    int64_t stride;             // floats from row to row
};

struct AttnArgs {
    KvArgs c;
    const float *q;
    int64_t q_stride;
    float *o;                   // [n_rows][nq * hd]
    float *part;                // workspace: partial results of a split
    void *rec;                  // workspace: (first slot, chunks) of each (sequence, pair)
    int nq, group;              // query heads; query heads per KV head
    float scale;
};

struct RouteArgs {
    const float *z, *bias;
    int32_t *ids;
    float *wts;
    int64_t n_rows;
    int n_exp, sigmoid, n_group, group_top, topk_group, topk, renorm;
    float scale;
};

struct PromptPlan {
    int64_t tiles;              // tile ids per KV head
    int n_split;                // splits of a tile over the cache's length
};
PromptPlan plan_prompt(int64_t n_rows, int n_seq, int nkv, int group);

// Launchers: a hipError_t value (0 = success).
int launch_kv_append(int kv_type, const AppendArgs &a, void *stream);
int launch_attn(int kv_type, const AttnArgs &a, void *stream);
int launch_attn_prompt(int kv_type, const AttnArgs &a, void *stream);
int launch_route(const RouteArgs &a, void *stream);

}  // namespace qg
