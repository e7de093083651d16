// bq_attn_bf16_split_shared.cu -- attention passes around shared pages of a bf16 cache, queries of other types (bq_attn.cuh).
#include "bq_attn.cuh"

BQ_ATTN_UNIT(bf16_split_shared, BQ_ATTN_INSTS(bq::KV_BF16, 3, 3, true),
             BQ_ATTN_INST(bq::KV_BF16, 3, 3, 64, 4, true), BQ_ATTN_INST(bq::KV_BF16, 3, 3, 128, 4, true))
