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
};

// work units of one request of n positions: at least one, which writes the rows
__host__ __device__ inline int attn_chunks(int n, int chunk) { return n <= chunk ? 1 : (n + chunk - 1) / chunk; }

struct AttnInstance {
    int dim, nt;  // head_dim up to dim, 8 nt query rows per CTA
    size_t smem;  // without the scan of the requests
    int (*occupancy)(size_t smem, int *out);
    cudaError_t (*launch)(const AttnArgs &, int grid, size_t smem, void *stream, unsigned int *status);
};

}  // namespace bq

// instance tables by cache type and split; n receives the number
const bq::AttnInstance *bq_internal_attn_f16_own(int *n);
const bq::AttnInstance *bq_internal_attn_f16_split(int *n);
const bq::AttnInstance *bq_internal_attn_bf16_own(int *n);
const bq::AttnInstance *bq_internal_attn_bf16_split(int *n);
const bq::AttnInstance *bq_internal_attn_q8_0_own(int *n);
const bq::AttnInstance *bq_internal_attn_q8_0_split(int *n);
