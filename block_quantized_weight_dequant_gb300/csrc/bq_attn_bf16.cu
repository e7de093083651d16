// bq_attn_bf16.cu -- paged attention over a bf16 cache (bq_attn.cuh).
#include <atomic>

#include "bq_attn.cuh"

BQ_ATTN_UNIT(bf16, bq::KV_BF16, 1, 2, 3, 3)
