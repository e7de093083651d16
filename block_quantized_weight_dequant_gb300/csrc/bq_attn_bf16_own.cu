// bq_attn_bf16_own.cu -- paged attention over a bf16 cache, bf16 queries (bq_attn.cuh).
#include <atomic>
#include <type_traits>

#include "bq_attn.cuh"

BQ_ATTN_UNIT(bf16_own, BQ_ATTN_INSTS(bf16_own, bq::KV_BF16, 1, 3),
             BQ_ATTN_INST(bf16_own, bq::KV_BF16, 1, 3, 64, 4), BQ_ATTN_INST(bf16_own, bq::KV_BF16, 1, 3, 128, 4))
