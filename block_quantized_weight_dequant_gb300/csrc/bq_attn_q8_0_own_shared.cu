// bq_attn_q8_0_own_shared.cu -- attention passes around shared pages of a Q8_0 cache, 16-bit queries (bq_attn.cuh).
#include "bq_attn.cuh"

BQ_ATTN_UNIT(q8_0_own_shared, BQ_ATTN_INSTS(bq::KV_Q8, 1, 2, true))
