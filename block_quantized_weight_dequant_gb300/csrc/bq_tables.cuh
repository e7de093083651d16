// bq_tables.cuh -- shared by the block tables of a step (bq_tables.cu) and those
// whose requests share pages (bq_pages.cu).
#pragma once

#include "bq_cache.cuh"

namespace bq {

struct RowsArgs {
    bq_kv_tables t;
    FastDiv page;
};

constexpr int TABLES_MAX_REQUESTS = 4096;
constexpr long long TABLES_ROWS_ALONE = 4096;  // token rows beyond which the slot map has a kernel of its own

// largest i in [0, n) with pre[i] <= x, for a non-decreasing pre with pre[0] <= x
__device__ __forceinline__ int last_not_above(const int *pre, int n, int x) {
    int lo = 0, hi = n;  // pre[lo] <= x, pre[hi] > x (or hi == n)
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pre[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

// what bqgemv.h says of bq_kv_tables
bq_status check_tables(const bq_kv_tables *t);
// the slot map from the finished table and the outputs, over the whole GPU
cudaError_t rows_launch(const bq_kv_tables &t, void *stream);

}  // namespace bq

int bq_internal_status_pages(unsigned int *flags, int clear);  // bq_pages.cu
