// bq_attn_f16_split_shared.cu -- attention passes around shared pages of an fp16 cache, queries of other types (bq_attn.cuh).
#include "bq_attn.cuh"

BQ_ATTN_UNIT(f16_split_shared, BQ_ATTN_INSTS(bq::KV_F16, 2, 2, true),
             BQ_ATTN_INST(bq::KV_F16, 2, 2, 64, 4, true), BQ_ATTN_INST(bq::KV_F16, 2, 2, 128, 4, true))
