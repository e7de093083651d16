// bq_attn_f16_split.cu -- paged attention over an fp16 cache, queries of other types (bq_attn.cuh).
#include <atomic>
#include <type_traits>

#include "bq_attn.cuh"

BQ_ATTN_UNIT(f16_split, BQ_ATTN_INSTS(f16_split, bq::KV_F16, 2, 2),
             BQ_ATTN_INST(f16_split, bq::KV_F16, 2, 2, 64, 4), BQ_ATTN_INST(f16_split, bq::KV_F16, 2, 2, 128, 4))
