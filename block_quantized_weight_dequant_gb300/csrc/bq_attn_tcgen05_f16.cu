// bq_attn_tcgen05_f16.cu -- shared pages of an fp16 cache (bq_attn_tcgen05.cuh).
#include "bq_attn_tcgen05.cuh"

cudaError_t bq_internal_prefix_f16(const bq::TcArgs &a, int grid, void *stream, unsigned int *status) {
    return a.a.x.dtype == BQ_F16 ? bq::prefix_launch<true, 1>(a, grid, stream, status)
                               : bq::prefix_launch<true, 2>(a, grid, stream, status);
}
