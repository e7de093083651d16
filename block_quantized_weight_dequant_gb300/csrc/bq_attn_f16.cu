// bq_attn_f16.cu -- paged attention over a f16 cache (bq_attn.cuh).
#include <atomic>

#include "bq_attn.cuh"

BQ_ATTN_UNIT(f16, bq::KV_F16, 1, 2, 2, 2)
