// attn_internal.h -- library-internal declarations of the attention side (paged key-value cache,
// attention, expert routing) shared by abi_attn.cpp and its kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace qg {

// Workgroup slots of the split over a cache's length (qgemv_attn): as many workgroups as are resident
// at once, two per compute unit up to head_dim 128 (8-wave registers), one above.  More, smaller
// chunks cost more than they balance: 64 x 7500 positions x 2 heads of 128 98.0 us with 512 slots and
// 102.9 with 768, 16 x 4000 x 4 heads of 256 53.6 with 256 and 62.2 with 512, 16 x 16000 x 8 heads of
// 64 90.2 with 512 and 99.5 with 1024.
#define ATTN_MAX_SLOTS 512
__host__ __device__ constexpr int attn_slots(int hd) { return hd <= 128 ? 512 : 256; }
// Floats of one slot's partial result: O of `cols` query heads, their exponents and sums.
__host__ __device__ constexpr int64_t attn_part_floats(int cols, int hd) { return (int64_t)cols * (hd + 2); }
// The same of qgemv_attn_prompt's 128-column tiles, and the most pairs of a call that may be split.
#define PROMPT_SLOTS 512
#define PROMPT_SPLITS 1024
__host__ __device__ constexpr int prompt_slots(int hd) { return hd <= 128 ? PROMPT_SLOTS : 256; }

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

struct PromptSplit;             // a split tile (attn_prompt_kernels.hip)

struct AttnArgs {
    KvArgs c;
    const float *q;
    int64_t q_stride;
    float *o;                   // [n_rows][nq * hd]
    float *part;                // workspace: partial results of a split
    int *pairs;                 // workspace: pairs of a prompt call
    PromptSplit *splits;        // workspace: its split tiles, by pair
    unsigned int *count;        // workspace: arrival counters of a split, one per slot, 0 between calls
    int nq, group;              // query heads; query heads per KV head
    int side;                   // set by the launcher: tiles that read the same positions
    float scale;
};

struct RouteArgs {
    const float *z, *bias;
    int32_t *ids;
    float *wts;
    int64_t n_rows;
    int n_exp, sigmoid, n_group, group_top, topk_group, topk, renorm;
    int run_log2;               // set by the launcher
    float scale;
};

struct PromptPlan {
    int64_t pairs;              // pairs of a tile and a KV head, at most
    int slots;                  // workgroup slots of a split over the cache's length, 0: none
    bool second;                // a second launch joins the parts
    int64_t grid;               // workgroups
};
PromptPlan plan_prompt(int64_t n_rows, int n_seq, int nkv, int group, int hd, int64_t positions);
bool prompt_in_16s(int64_t n_rows, int n_seq, int nq, int nkv, int hd, int64_t positions);

// Launchers: a hipError_t value (0 = success).
int launch_kv_append(int kv_type, const AppendArgs &a, void *stream);
int launch_attn(int kv_type, const AttnArgs &a, void *stream);
int launch_attn_rows(int kv_type, const AttnArgs &a, void *stream);     // few rows per sequence
int launch_attn_prompt(int kv_type, const AttnArgs &a, void *stream);
int launch_route(const RouteArgs &a, void *stream);

}  // namespace qg
