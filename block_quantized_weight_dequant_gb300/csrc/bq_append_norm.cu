// bq_append_norm.cu -- the append with norms of queries and keys (bq_append.cuh).
#include "bq_append.cuh"

cudaError_t bq::append_normed(const AppendArgs &a, int grid, void *stream, unsigned int *status) {
    return append_launch<true>(a, grid, stream, status);
}
