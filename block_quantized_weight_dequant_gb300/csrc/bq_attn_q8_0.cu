// bq_attn_q8_0.cu -- paged attention over a q8_0 cache (bq_attn.cuh).
#include <atomic>

#include "bq_attn.cuh"

BQ_ATTN_UNIT(q8_0, bq::KV_Q8, 1, 2, 3, 3)
