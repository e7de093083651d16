// bq_attn_f16_own_shared.cu -- attention passes around shared pages of an fp16 cache, fp16 queries (bq_attn.cuh).
#include "bq_attn.cuh"

BQ_ATTN_UNIT(f16_own_shared, BQ_ATTN_INSTS(bq::KV_F16, 1, 2, true),
             BQ_ATTN_INST(bq::KV_F16, 1, 2, 64, 4, true), BQ_ATTN_INST(bq::KV_F16, 1, 2, 128, 4, true))
