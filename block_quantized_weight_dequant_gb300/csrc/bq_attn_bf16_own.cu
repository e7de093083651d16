// bq_attn_bf16_own.cu -- paged attention over a bf16 cache, bf16 queries (bq_attn.cuh).
#include "bq_attn.cuh"

BQ_ATTN_UNIT(bf16_own, BQ_ATTN_INSTS(bq::KV_BF16, 1, 3),
             BQ_ATTN_INST(bq::KV_BF16, 1, 3, 64, 4), BQ_ATTN_INST(bq::KV_BF16, 1, 3, 128, 4))
