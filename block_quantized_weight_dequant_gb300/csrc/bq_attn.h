// bq_attn.h -- arguments and instances of the paged attention kernels, shared
// by the planner (bq_attn.cu) and the instance units (bq_attn_<cache>.cu).
#pragma once

#include <cstddef>
#include <cstdint>

#include "bq_cache.cuh"

namespace bq {

constexpr int ATTN_WARPS = 4;
constexpr int ATTN_CLUSTER = 8;  // most chunks that a cluster joins
constexpr int ATTN_MAX_REQUESTS = 4096;
// softmax weights are 2^(s - max + SHIFT): with fp16 parts this keeps weights
// down to 2^-29 of the largest in fp16's normal range; the sum of the weights
// carries the same factor, so it cancels
constexpr int ATTN_SHIFT_F16 = 15;

// What a launch of the attention kernel covers.  ATTN_REST and ATTN_PREFIX write
// partial results alone, which a join of their own puts together (bq_attn_prefix.cu).
enum {
    ATTN_ALL = 0,    // all positions of each request
    ATTN_REST = 1,   // the positions behind the pages that a group of requests shares
    ATTN_PREFIX = 2, // the shared pages: "requests" are groups, whose rows are all rows of their requests
    ATTN_WHOLE = 3   // as ATTN_ALL, but nothing for requests that do not see their shared pages
};
constexpr int ATTN_GROUPS = BQ_PREFIX_MAX_GROUPS;

struct AttnArgs {
    bq_kv_cache c;
    bq_attention_args x;
    FastDiv page;
    FastDiv group;
    int group_rows;  // query rows of one kv head: heads / kv_heads * rows
    int row_tiles;   // tiles of 8 NT query rows
    int chunk;       // positions of a work unit
    int max_chunks;  // units of the longest request the table can hold
    int direct;      // a CTA for every unit that the table can hold
    int cluster;     // a request's max_chunks units are a cluster, which joins them
    float scale_log2;
    float *part_o;   // [unit][8 NT rows][head_dim] unnormalised, with max_chunks > 1
    float2 *part_ml; // [unit][8 NT rows] running maximum and sum
    int mode;        // ATTN_ALL, or:
    int group_end[ATTN_GROUPS];    // requests up to the end of each group
    int group_pages[ATTN_GROUPS];  // whole pages that its requests share
};

// a request's length, of which the table holds `most` (a difference of one as it was
// given may pass 2^31)
__host__ __device__ inline int attn_clamped(int len, int most) { return len < 0 ? 0 : len < most ? len : most; }
// whether a request's rows see all of `shared` positions, from its clamped length (none
// are seen by a request shorter than its rows, too)
__host__ __device__ inline bool attn_sees(int len, int rows, int shared) {
    return shared == 0 || len - rows + 1 >= shared;
}
// positions that its rows see behind them: none unless they see the shared ones
__host__ __device__ inline int attn_rest(int len, int rows, int shared) {
    return attn_sees(len, rows, shared) ? len - shared : 0;
}

// work units of one request of n positions: at least one, which writes the rows
__host__ __device__ inline int attn_chunks(int n, int chunk) { return n <= chunk ? 1 : (n + chunk - 1) / chunk; }

// positions that an ATTN_ALL or ATTN_WHOLE launch sees of request b
__device__ inline int attn_length(const AttnArgs &a, int b) {
    const int n = attn_clamped(a.x.lens[b], a.x.table_width * a.c.page_size);
    if (a.mode == ATTN_ALL) return n;
    int g = 0;
    while (a.group_end[g] <= b) ++g;
    return attn_sees(n, a.x.rows, a.group_pages[g] * a.c.page_size) ? n : 0;
}

struct AttnInstance {
    int dim, nt;  // head_dim up to dim, 8 nt query rows per CTA
    size_t smem;  // without the scan of the requests
    int (*occupancy)(size_t smem, int *out);
    cudaError_t (*launch)(const AttnArgs &, int grid, size_t smem, void *stream, unsigned int *status);
};

// what bqgemv.h says of bq_attention_args: shapes, then pointers (and the cache's)
bq_status check_attention_shape(const bq_kv_cache *c, const bq_attention_args *x);
bq_status check_attention_pointers(const bq_kv_cache *c, const bq_attention_args *x);
// the instance that serves the call's types with nt n-tiles, in ATTN_ALL or another
// mode, NULL if there is none
const AttnInstance *attn_instance(const bq_kv_cache *c, int dtype, int nt, bool modes);
// n-tiles for a number of query rows of a kv head
int attn_tiles(const bq_kv_cache *c, int64_t group_rows);

}  // namespace bq

// instance tables by cache type and split; n receives the number
const bq::AttnInstance *bq_internal_attn_f16_own(int *n);
const bq::AttnInstance *bq_internal_attn_f16_own_shared(int *n);
const bq::AttnInstance *bq_internal_attn_f16_split(int *n);
const bq::AttnInstance *bq_internal_attn_f16_split_shared(int *n);
const bq::AttnInstance *bq_internal_attn_bf16_own(int *n);
const bq::AttnInstance *bq_internal_attn_bf16_own_shared(int *n);
const bq::AttnInstance *bq_internal_attn_bf16_split(int *n);
const bq::AttnInstance *bq_internal_attn_bf16_split_shared(int *n);
const bq::AttnInstance *bq_internal_attn_q8_0_own(int *n);
const bq::AttnInstance *bq_internal_attn_q8_0_own_shared(int *n);
const bq::AttnInstance *bq_internal_attn_q8_0_split(int *n);
const bq::AttnInstance *bq_internal_attn_q8_0_split_shared(int *n);

// bq_attn.cu: the call in one pass, with the groups of `shared` (or NULL)
bq_status bq_internal_paged_attention(const bq_kv_cache *cache, const bq_attention_args *x, const bq::AttnArgs *shared,
                                      void *workspace, int64_t workspace_bytes, void *stream);
