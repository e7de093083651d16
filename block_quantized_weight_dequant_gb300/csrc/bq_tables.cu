// bq_tables.cu -- block tables, slot map and free pages of a step, built on
// the GPU from the requests' lengths (bq_kv_block_tables in include/bqgemv.h).
//
// One thread-block cluster builds tables, free stack and lengths.  Every CTA
// reads the lengths and scans, over the requests, the pages released, the pages
// asked and the token rows (three prefix sums of at most 4096 numbers, kept in
// its shared memory, so no CTA waits for another's scan).  The cluster passes
// one barrier before lens_out and free_count_out are written, after which
// nobody reads the lengths or the count again: they may be the inputs.
//   released page i -> stack[free + i], pushed before anything is popped
//   asked page i    <- stack[free + released - 1 - i]
// so an asked page is either one of the released ones (found by a search of the
// released prefix sums, read from the table row it leaves) or an old entry of
// the stack, and a pushed page that is popped again is never written.  The
// entries read (rows that shrink, the stack below the old top) and written
// (rows that grow, the stack above it) are apart, so the order of threads
// does not matter.  Nothing is accumulated with atomics.
// The slot map of few rows is written by the same launch; of many by a second
// kernel over the whole GPU, which reads the finished table.  What a row needs
// of its request follows from the outputs: a request is served if lens_out is
// new_lens, and grew by its number of rows.  Bound by latency: 256 requests of a
// decode step 7.0 us, 1000 with prompts (92000 rows) 11.5 us.
#include "bq_tables.cuh"

namespace {

BQ_STATUS_WORD(tables)

constexpr int THREADS = 512;
constexpr int MAX_CLUSTER = 8;

using Args = bq::RowsArgs;

struct Request {
    int lo, hi;          // lengths before and after; equal for a request that is left alone
    int held, wanted;    // pages
    bool bad;            // a length out of range
};

__device__ __forceinline__ Request request_of(const Args &a, int lo, int hi) {
    const long long most = (long long)a.t.table_width * a.t.page_size;
    Request r;
    r.bad = lo < 0 || hi < 0 || lo > most || hi > most;
    r.lo = lo;
    r.hi = r.bad ? lo : hi;
    // n + page_size - 1 may pass 2^31: divide n and add one for a remainder
    auto pages = [&](int n) {
        const uint32_t q = a.page.div((uint32_t)n);
        return (int)(q + ((uint32_t)n - q * a.page.d != 0));
    };
    r.held = r.bad ? 0 : pages(lo);
    r.wanted = r.bad ? 0 : pages(hi);
    return r;
}

__global__ void __launch_bounds__(THREADS) tables_kernel(const __grid_constant__ Args a, int with_rows) {
    extern __shared__ int sm[];
    const int n = a.t.requests, tid = threadIdx.x;
    int *freed = sm, *asked = sm + (n + 1), *rows = sm + 2 * (n + 1);  // exclusive prefix sums
    int *lo_s = sm + 3 * (n + 1), *hi_s = lo_s + n;                    // lengths as read
    __shared__ long long warp_sums[3][THREADS / 32];
    __shared__ int s_given, s_refused;
    bq::pdl_wait();
    if (!with_rows) bq::pdl_launch_dependents();
    uint32_t rank, cluster;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(cluster));
    if (tid == 0) s_given = s_refused = 0;
    const int count_in = *a.t.free_count;
    for (int b = tid; b < n; b += THREADS) {
        lo_s[b] = a.t.lens[b];
        hi_s[b] = a.t.new_lens[b];
    }
    __syncthreads();
    auto request = [&](int b) { return request_of(a, lo_s[b], hi_s[b]); };

    // each thread sums a contiguous run of requests, then the runs are scanned
    const int per = (n + THREADS - 1) / THREADS;
    const int b0 = min(n, tid * per), b1 = min(n, b0 + per);
    long long sum[3] = {0, 0, 0};
    for (int b = b0; b < b1; ++b) {
        const Request r = request(b);
        sum[0] += max(0, r.held - r.wanted);
        sum[1] += max(0, r.wanted - r.held);
        sum[2] += max(0, r.hi - r.lo);
    }
    long long excl[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        long long v = sum[k];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(~0u, v, o);
            if ((tid & 31) >= o) v += u;
        }
        if ((tid & 31) == 31) warp_sums[k][tid >> 5] = v;
        excl[k] = v - sum[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 3; ++k)
        for (int w = 0; w < (tid >> 5); ++w) excl[k] += warp_sums[k][w];
    // Sums are clamped to 2^31 - 1, which is more than any pool or max_tokens
    // holds, so a clamped sum decides as the true one does.
    const long long TOP = 0x7fffffffLL;
    for (int b = b0; b < b1; ++b) {
        const Request r = request(b);
        freed[b] = (int)min(TOP, excl[0]);
        asked[b] = (int)min(TOP, excl[1]);
        rows[b] = (int)min(TOP, excl[2]);
        excl[0] += max(0, r.held - r.wanted);
        excl[1] += max(0, r.wanted - r.held);
        excl[2] += max(0, r.hi - r.lo);
    }
    if (b1 == n && b0 < n) {  // the thread with the last request
        freed[n] = (int)min(TOP, excl[0]);
        asked[n] = (int)min(TOP, excl[1]);
        rows[n] = (int)min(TOP, excl[2]);
    }
    if (n == 0 && tid == 0) freed[0] = asked[0] = rows[0] = 0;
    __syncthreads();

    const int pool = a.t.pool;
    const int count = min(max(count_in, 0), pool);
    int released = freed[n];
    const bool over = count_in != count || released > pool - count;
    released = min(released, pool - count);
    if (over && tid == 0 && rank == 0) atomicOr(&g_status_tables, BQ_DEVERR_POOL);
    const int avail = count + released;
    auto served = [&](int b, const Request &r) {
        return !r.bad && (r.wanted <= r.held || asked[b + 1] <= avail) &&
               (r.hi <= r.lo || rows[b + 1] <= a.t.max_tokens);
    };
    // the i-th asked page
    auto page_at = [&](int i) {
        const int at = avail - 1 - i;
        if (at < count) return a.t.free_pages[at];
        const int b = bq::last_not_above(freed, n, at - count);
        return a.t.table[b * a.t.table_stride + request(b).wanted + (at - count - freed[b])];
    };

    int given = 0, refused = 0;
    for (int b = tid; b < n; b += THREADS) {
        const Request r = request(b);
        const bool ok = served(b, r);
        if (ok && r.wanted > r.held) given = max(given, asked[b + 1]);
        refused += !ok;
    }
    given = __reduce_max_sync(~0u, given);
    refused = __reduce_add_sync(~0u, refused);
    if ((tid & 31) == 0) {
        atomicMax(&s_given, given);
        atomicAdd(&s_refused, refused);
    }
    __syncthreads();
    given = s_given;

    // pages: one asked or pushed entry per thread
    const int step = (int)cluster * THREADS, first = (int)rank * THREADS + tid;
    for (int i = first; i < given; i += step) {
        const int page = page_at(i);
        const int b = bq::last_not_above(asked, n, i);
        a.t.table[b * a.t.table_stride + request(b).held + (i - asked[b])] = page;
    }
    for (int i = first; i < released - given; i += step) {
        const int b = bq::last_not_above(freed, n, i);
        a.t.free_pages[count + i] = a.t.table[b * a.t.table_stride + request(b).wanted + (i - freed[b])];
    }
    if (with_rows) {
        // the page of a token is an old entry of its row or the asked page that the
        // loop above writes there, taken from its source
        const long long total = min((long long)rows[n], (long long)a.t.max_tokens);
        for (long long t = first; t < a.t.max_tokens; t += step) {
            long long slot = -1;
            int position = 0;
            if (t < total) {
                const int b = bq::last_not_above(rows, n, (int)t);
                const Request r = request(b);
                if (served(b, r)) {
                    position = r.lo + (int)(t - rows[b]);
                    const int q = (int)a.page.div((uint32_t)position);
                    const int page = q < r.held ? a.t.table[b * a.t.table_stride + q] : page_at(asked[b] + q - r.held);
                    slot = (long long)page * a.t.page_size + (position - q * a.t.page_size);
                }
            }
            a.t.slots[t] = slot;
            a.t.positions[t] = position;
        }
    }
    for (int b = first; b <= n; b += step) a.t.starts[b] = rows[b];

    // every CTA has read the lengths and the count: now they may be overwritten
    if (cluster > 1) {
        asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    } else {
        __syncthreads();
    }
    for (int b = first; b < n; b += step) {
        const Request r = request(b);
        a.t.lens_out[b] = served(b, r) ? r.hi : r.lo;
    }
    if (rank == 0 && tid == 0) {
        *a.t.free_count_out = avail - given;
        *a.t.refused = s_refused;
    }
}

}  // namespace

namespace bq {

constexpr int ROWS_THREADS = 256, ROWS_EACH = 4;  // tokens per thread

// the slot map from the finished table: a few tokens per thread
__global__ void __launch_bounds__(ROWS_THREADS) rows_kernel(const __grid_constant__ RowsArgs a) {
    extern __shared__ int starts[];
    const int n = a.t.requests;
    const long long t0 = ((long long)blockIdx.x * ROWS_THREADS + threadIdx.x) * ROWS_EACH;
    pdl_wait();
    for (int b = threadIdx.x; b <= n; b += ROWS_THREADS) starts[b] = a.t.starts[b];
    __syncthreads();
    const long long total = min((long long)starts[n], (long long)a.t.max_tokens);
    int b = t0 < total ? last_not_above(starts, n, (int)t0) : 0;
    long long slot[ROWS_EACH];
    int position[ROWS_EACH];
#pragma unroll
    for (int i = 0; i < ROWS_EACH; ++i) {
        const long long t = t0 + i;
        slot[i] = -1;
        position[i] = 0;
        if (t < total) {
            while (starts[b + 1] <= t) ++b;  // ends: starts[n] > t
            const int hi = a.t.new_lens[b];
            if (a.t.lens_out[b] == hi) {
                position[i] = hi - (starts[b + 1] - (int)t);
                const int q = (int)a.page.div((uint32_t)position[i]);
                slot[i] = (long long)a.t.table[b * a.t.table_stride + q] * a.t.page_size +
                          (position[i] - q * a.t.page_size);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < ROWS_EACH; ++i)
        if (t0 + i < a.t.max_tokens) {
            a.t.slots[t0 + i] = slot[i];
            a.t.positions[t0 + i] = position[i];
        }
}

bq_status check_tables(const bq_kv_tables *t) {
    if (!t) return BQ_ERR_NULL;
    if (t->requests < 0 || t->requests > TABLES_MAX_REQUESTS || t->page_size < 1 || t->page_size > 65536 ||
        t->table_width < 1 || t->table_stride < t->table_width || t->table_stride > (1LL << 40) ||
        t->max_tokens < 0 || t->max_tokens > 0x7ffffffeLL || t->pool < 1 || t->pool == 0x7fffffff)
        return BQ_ERR_SHAPE;
    // the slot map is made from the lengths asked and the lengths given
    if (t->requests && t->lens_out && t->lens_out == t->new_lens) return BQ_ERR_SHAPE;
    const void *need[] = {t->free_pages, t->free_count, t->starts, t->free_count_out, t->refused};
    for (const void *p : need)
        if (!p) return BQ_ERR_NULL;
    if (t->requests && (!t->lens || !t->new_lens || !t->table || !t->lens_out)) return BQ_ERR_NULL;
    if (t->max_tokens && (!t->slots || !t->positions)) return BQ_ERR_NULL;
    const void *words[] = {t->lens, t->new_lens, t->table, t->free_pages, t->free_count, t->positions,
                           t->starts, t->lens_out, t->free_count_out, t->refused};
    for (const void *p : words)
        if (!aligned_to(p, 4)) return BQ_ERR_ALIGN;
    if (!aligned_to(t->slots, 8)) return BQ_ERR_ALIGN;
    return BQ_OK;
}

cudaError_t rows_launch(const bq_kv_tables &t, void *stream) {
    RowsArgs a;
    a.t = t;
    a.page.set((uint32_t)t.page_size);
    const long long per_cta = (long long)ROWS_THREADS * ROWS_EACH;
    return launch_pdl(rows_kernel, dim3((unsigned)((t.max_tokens + per_cta - 1) / per_cta)), ROWS_THREADS,
                      (size_t)(t.requests + 1) * sizeof(int), stream, 1, a);
}

}  // namespace bq

int bq_internal_status_tables(unsigned int *flags, int clear) {
    unsigned int a = 0, b = 0;
    int e = read_status_tables(&a, clear);
    if (e == 0) e = bq_internal_status_pages(&b, clear);
    *flags = a | b;
    return e;
}

extern "C" bq_status bq_kv_block_tables(const bq_kv_tables *t, void *stream) {
    const bq_status s = bq::check_tables(t);
    if (s != BQ_OK) return s;
    Args a;
    a.t = *t;
    a.page.set((uint32_t)t->page_size);
    // One launch for few rows (a decode step), two for many (1000 requests with
    // 92000 rows of prompts: 11.6 us, 41 us in one launch of 8 CTAs).
    const bool with_rows = t->max_tokens <= bq::TABLES_ROWS_ALONE;
    // CTAs for the pages that may be asked, each of its threads a few
    const long long work = (with_rows ? t->max_tokens : t->max_tokens / t->page_size) + t->requests;
    int cluster = 1;
    while (cluster < MAX_CLUSTER && work > 2LL * THREADS * cluster) cluster *= 2;
    const size_t smem = (size_t)(5 * (t->requests + 1)) * sizeof(int);
    if (smem > 47 * 1024) {  // (400 bytes of static shared memory count against the 48 KB too)
        const cudaError_t e = cudaFuncSetAttribute(tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)(5 * (bq::TABLES_MAX_REQUESTS + 1) * sizeof(int)));
        if (e != cudaSuccess) return bq::from_cuda_error(e);
    }
    cudaError_t e = bq::launch_pdl(tables_kernel, dim3((unsigned)cluster), THREADS, smem, stream, cluster, a,
                                   (int)with_rows);
    if (e != cudaSuccess || with_rows) return bq::from_cuda_error(e);
    return bq::from_cuda_error(bq::rows_launch(a.t, stream));
}
