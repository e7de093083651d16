// bq_attn_q8_0_split.cu -- paged attention over a Q8_0 cache, queries of other types (bq_attn.cuh).
#include "bq_attn.cuh"

BQ_ATTN_UNIT(q8_0_split, BQ_ATTN_INSTS(bq::KV_Q8, 2, 2))
