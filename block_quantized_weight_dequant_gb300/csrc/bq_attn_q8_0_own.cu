// bq_attn_q8_0_own.cu -- paged attention over a Q8_0 cache, 16-bit queries (bq_attn.cuh).
#include "bq_attn.cuh"

BQ_ATTN_UNIT(q8_0_own, BQ_ATTN_INSTS(bq::KV_Q8, 1, 2, false))
