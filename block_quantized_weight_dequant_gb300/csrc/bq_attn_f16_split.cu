// bq_attn_f16_split.cu -- paged attention over an fp16 cache, queries of other types (bq_attn.cuh).
#include "bq_attn.cuh"

BQ_ATTN_UNIT(f16_split, BQ_ATTN_INSTS(bq::KV_F16, 2, 2, false),
             BQ_ATTN_INST(bq::KV_F16, 2, 2, 64, 4, false), BQ_ATTN_INST(bq::KV_F16, 2, 2, 128, 4, false))
