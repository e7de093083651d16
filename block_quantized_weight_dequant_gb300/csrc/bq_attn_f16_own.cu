// bq_attn_f16_own.cu -- paged attention over an fp16 cache, fp16 queries (bq_attn.cuh).
#include <atomic>
#include <type_traits>

#include "bq_attn.cuh"

BQ_ATTN_UNIT(f16_own, BQ_ATTN_INSTS(f16_own, bq::KV_F16, 1, 2),
             BQ_ATTN_INST(f16_own, bq::KV_F16, 1, 2, 64, 4), BQ_ATTN_INST(f16_own, bq::KV_F16, 1, 2, 128, 4))
