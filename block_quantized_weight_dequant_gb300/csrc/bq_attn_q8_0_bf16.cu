// bq_attn_q8_0_bf16.cu -- paged attention over a Q8_0 cache, bf16 queries (bq_attn.cuh).
#include <atomic>
#include <type_traits>

#include "bq_attn.cuh"

BQ_ATTN_UNIT(q8_0_bf16, BQ_ATTN_INSTS(q8_0_bf16, bq::KV_Q8, 1, 1))
