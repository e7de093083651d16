// bq_attn_f16_own.cu -- paged attention over an fp16 cache, fp16 queries (bq_attn.cuh).
#include "bq_attn.cuh"

BQ_ATTN_UNIT(f16_own, BQ_ATTN_INSTS(bq::KV_F16, 1, 2),
             BQ_ATTN_INST(bq::KV_F16, 1, 2, 64, 4), BQ_ATTN_INST(bq::KV_F16, 1, 2, 128, 4))
