// bq_attn_tcgen05_bf16.cu -- shared pages of a bf16 cache (bq_attn_tcgen05.cuh).
#include "bq_attn_tcgen05.cuh"

cudaError_t bq_internal_prefix_bf16(const bq::TcArgs &a, int grid, void *stream, unsigned int *status) {
    return a.a.x.dtype == BQ_BF16 ? bq::prefix_launch<false, 1>(a, grid, stream, status)
                                : bq::prefix_launch<false, 3>(a, grid, stream, status);
}
