// bq_attn_bf16_split.cu -- paged attention over a bf16 cache, queries of other types (bq_attn.cuh).
#include "bq_attn.cuh"

BQ_ATTN_UNIT(bf16_split, BQ_ATTN_INSTS(bq::KV_BF16, 3, 3, false),
             BQ_ATTN_INST(bq::KV_BF16, 3, 3, 64, 4, false), BQ_ATTN_INST(bq::KV_BF16, 3, 3, 128, 4, false))
