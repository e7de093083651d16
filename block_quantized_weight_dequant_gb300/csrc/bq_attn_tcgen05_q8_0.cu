// bq_attn_tcgen05_q8_0.cu -- shared pages of a Q8_0 cache (bq_attn_tcgen05.cuh).
#include "bq_attn_tcgen05.cuh"

cudaError_t bq_internal_prefix_q8_0(const bq::TcArgs &a, int grid, void *stream, unsigned int *status) {
    return a.a.x.dtype == BQ_F32 ? bq::prefix_launch<true, 2, true>(a, grid, stream, status)
                                 : bq::prefix_launch<true, 1, true>(a, grid, stream, status);
}
