// bq_attn.cu -- planning of the paged attention and the join of its chunks
// (bq_paged_attention in include/bqgemv.h; the kernel is bq_attn.cuh).
#include <atomic>
#include <cmath>

#include "bq_attn.h"

int bq_internal_status_attn_prefix(unsigned int *flags, int clear);  // bq_attn_prefix.cu

namespace {

BQ_STATUS_WORD(attn)

// the status word's device address, looked up once per device
cudaError_t status_address(unsigned int **out) {
    static std::atomic<unsigned int *> addr[64];
    return bq::symbol_address(addr, g_status_attn, out);
}

constexpr int JOIN_THREADS = 256;

// Joins a request's chunks: one CTA per query row and head.  Chunk i's weight
// is 2^(m_i - max m); the chunks are taken by thread groups of D / 4 lanes in a
// fixed order.  A request of one chunk was written by the attention kernel.
template <int DT>
__global__ void __launch_bounds__(JOIN_THREADS) join_kernel(const __grid_constant__ bq::AttnArgs a, int tile_rows) {
    extern __shared__ float w_s[];  // [max_chunks] weights, then [groups][D] partial sums
    __shared__ float red[2][JOIN_THREADS / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int D = a.c.head_dim, R = a.x.rows;
    const int head = blockIdx.x % a.x.heads;
    const int token = blockIdx.x / a.x.heads;  // request * rows + row
    const int b = token / R, row = token - b * R;
    const int h = (int)a.group.div((uint32_t)head);
    const int g = row * (int)a.group.d + head - h * (int)a.group.d;
    const int rt = g / tile_rows, i = g - rt * tile_rows;
    bq::pdl_wait();
    const int chunks = bq::attn_chunks(bq::attn_length(a, b), a.chunk);
    if (chunks == 1) return;
    const long long unit0 = (((long long)b * a.max_chunks) * a.c.kv_heads + h) * a.row_tiles + rt;
    const long long step = (long long)a.c.kv_heads * a.row_tiles;
    const int vecs = D / 4, groups = JOIN_THREADS / vecs;  // D <= 256: at least four groups
    const int gr = tid / vecs, v = tid - gr * vecs;
    const float *src = a.part_o + (unit0 * tile_rows + i) * D + 4 * v;
    const long long hop = step * tile_rows * D;
    // the first AHEAD partial sums of this thread while the weights are computed
    constexpr int AHEAD = 8;
    float4 first[AHEAD];
#pragma unroll
    for (int x = 0; x < AHEAD; ++x) {
        const int k = gr + x * groups;
        if (gr < groups && k < chunks) first[x] = *reinterpret_cast<const float4 *>(src + k * hop);
    }
    float top = -INFINITY;
    for (int k = tid; k < chunks; k += JOIN_THREADS)
        top = fmaxf(top, a.part_ml[(unit0 + k * step) * tile_rows + i].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    if (lane == 0) red[0][warp] = top;
    __syncthreads();
    for (int w = 0; w < JOIN_THREADS / 32; ++w) top = fmaxf(top, red[0][w]);
    float sum = 0.0f;
    for (int k = tid; k < chunks; k += JOIN_THREADS) {
        const float2 ml = a.part_ml[(unit0 + k * step) * tile_rows + i];
        const float f = ml.x == -INFINITY ? 0.0f : exp2f(ml.x - top);
        w_s[k] = f;
        sum = fmaf(f, ml.y, sum);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    if (lane == 0) red[1][warp] = sum;
    __syncthreads();
    sum = 0.0f;
    for (int w = 0; w < JOIN_THREADS / 32; ++w) sum += red[1][w];

    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    auto add = [&](int k, const float4 &o) {
        const float f = w_s[k];
        acc.x = fmaf(f, o.x, acc.x);
        acc.y = fmaf(f, o.y, acc.y);
        acc.z = fmaf(f, o.z, acc.z);
        acc.w = fmaf(f, o.w, acc.w);
    };
    if (gr < groups) {
#pragma unroll
        for (int x = 0; x < AHEAD; ++x)
            if (gr + x * groups < chunks) add(gr + x * groups, first[x]);
#pragma unroll 8
        for (int k = gr + AHEAD * groups; k < chunks; k += groups)
            add(k, *reinterpret_cast<const float4 *>(src + k * hop));
    }
    float *sums = w_s + (a.max_chunks + 3) / 4 * 4;
    if (gr < groups) *reinterpret_cast<float4 *>(sums + gr * D + 4 * v) = acc;
    __syncthreads();
    const long long at = (long long)token * a.x.out_row_stride + (long long)head * a.x.out_head_stride;
    for (int d = tid; d < D; d += JOIN_THREADS) {
        float o = 0.0f;
        for (int k = 0; k < groups; ++k) o += sums[k * D + d];
        o = sum == 0.0f ? 0.0f : o / sum;  // a row that sees nothing
        if constexpr (DT == BQ_F32) ((float *)a.x.out)[at + d] = o;
        else if constexpr (DT == BQ_F16) ((__half *)a.x.out)[at + d] = __float2half_rn(o);
        else ((__nv_bfloat16 *)a.x.out)[at + d] = __float2bfloat16_rn(o);
    }
}

// The same for tables of few chunks: a warp per query row and head, its lanes'
// four elements at a time, the chunks in order.
template <int DT>
__global__ void __launch_bounds__(JOIN_THREADS) join_few_kernel(const __grid_constant__ bq::AttnArgs a, int tile_rows) {
    const int lane = threadIdx.x & 31;
    const int index = (int)((blockIdx.x * JOIN_THREADS + threadIdx.x) >> 5);
    const int D = a.c.head_dim, R = a.x.rows;
    const int token = index / a.x.heads, head = index - token * a.x.heads;
    const int b = token / R, row = token - b * R;
    const int h = (int)a.group.div((uint32_t)head);
    const int g = row * (int)a.group.d + head - h * (int)a.group.d;
    const int rt = g / tile_rows, i = g - rt * tile_rows;
    bq::pdl_wait();
    if (b >= a.x.requests) return;
    const int chunks = bq::attn_chunks(bq::attn_length(a, b), a.chunk);
    if (chunks == 1) return;
    const long long unit0 = (((long long)b * a.max_chunks) * a.c.kv_heads + h) * a.row_tiles + rt;
    const long long step = (long long)a.c.kv_heads * a.row_tiles;
    const float *src = a.part_o + (unit0 * tile_rows + i) * D;
    const long long hop = step * tile_rows * D;
    const float2 ml = lane < chunks ? a.part_ml[(unit0 + lane * step) * tile_rows + i] : make_float2(-INFINITY, 0.0f);
    float top = ml.x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    const float f = ml.x == -INFINITY ? 0.0f : exp2f(ml.x - top);
    float sum = f * ml.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    const long long at = (long long)token * a.x.out_row_stride + (long long)head * a.x.out_head_stride;
    for (int d0 = 0; d0 < D; d0 += 128) {
        const int d = d0 + 4 * lane;
        const bool mine = d < D;
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
        for (int k = 0; k < chunks; ++k) {
            const float w = __shfl_sync(~0u, f, k);
            const float4 o = mine ? *reinterpret_cast<const float4 *>(src + k * hop + d) : acc;
            acc.x = fmaf(w, o.x, acc.x);
            acc.y = fmaf(w, o.y, acc.y);
            acc.z = fmaf(w, o.z, acc.z);
            acc.w = fmaf(w, o.w, acc.w);
        }
        if (mine) {
            const float v[4] = {acc.x, acc.y, acc.z, acc.w};
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const float y = sum == 0.0f ? 0.0f : v[x] / sum;  // a row that sees nothing
                if constexpr (DT == BQ_F32) ((float *)a.x.out)[at + d + x] = y;
                else if constexpr (DT == BQ_F16) ((__half *)a.x.out)[at + d + x] = __float2half_rn(y);
                else ((__nv_bfloat16 *)a.x.out)[at + d + x] = __float2bfloat16_rn(y);
            }
        }
    }
}

template <int DT>
cudaError_t join(const bq::AttnArgs &a, int tile_rows, void *stream) {
    const int64_t rows = (int64_t)a.x.requests * a.x.rows * a.x.heads;
    // up to 16 chunks a warp joins a row (160 requests of 14 heads, two chunks at
    // most: the call 30 us against 33 with a CTA per row), beyond it a CTA
    constexpr int JOIN_FEW = 16;
    if (a.max_chunks <= JOIN_FEW) {
        constexpr int PER = JOIN_THREADS / 32;
        return bq::launch_pdl(join_few_kernel<DT>, dim3((unsigned)((rows + PER - 1) / PER)), JOIN_THREADS, 0, stream, 1,
                              a, tile_rows);
    }
    const int groups = JOIN_THREADS / (a.c.head_dim / 4);
    const size_t smem = ((size_t)(a.max_chunks + 3) / 4 * 4 + (size_t)groups * a.c.head_dim) * sizeof(float);
    return bq::launch_pdl(join_kernel<DT>, dim3((unsigned)rows), JOIN_THREADS, smem, stream, 1, a, tile_rows);
}

struct Plan {
    const bq::AttnInstance *inst;
    bq::AttnArgs a;
    size_t smem;
    int64_t units;  // most units that the table can hold
    int64_t o_bytes, ml_bytes;
};

// Positions per work unit and how units are joined, from the geometry alone
// (not the query rows, so that every number of rows shares one order of sums).
//  - Where 8 units per request and kv head fit the GPU at once and are at most
//    CLUSTER_CHUNK positions long, they are clusters that join themselves: one
//    launch for two (16 heads over 4, fp16, 1000 positions: 7.0 us against 7.3;
//    at 4000, chunks of 512, 11.6 against 8.4).
//  - Else the table's capacity is cut into about TARGET units (two CTAs per SM,
//    one wave), 128 positions at least (two tiles per warp) and 2048 at most (so
//    that the longest table, 2^23 positions, has 4096 units, whose weights the
//    join keeps in shared memory).  Finer units for ragged requests cost more in
//    starts and joins than they balance (8 requests to 30000, 2 kv heads: 74 us
//    against 82, 77 and 82 with two, four and eight times the units; 16 to 4000, 8 kv
//    heads: 38 against 43, 44, 49).
// The table's capacity cuts, not the lengths, which the host does not know: a
// request in a table much wider than itself has few units (one request of 16 heads
// over 4, fp16: 700 positions 6.9 us in a table of their own, 11.5 in one of 32768,
// 12.6 in one of 131072; 8000 positions 8.6, 11.7, 26.0; 32768 in one of 131072 28.3
// against 18.8).
constexpr int64_t TARGET = 304, CHUNK_MIN = 128, CHUNK_MAX = 2048, CLUSTER_CHUNK = 256;
struct Chunking {
    int chunk;
    bool cluster;
};
Chunking chunking_of(int64_t requests, int64_t kv_heads, int64_t capacity) {
    const int64_t pairs = requests * kv_heads;
    int64_t n = ((capacity + bq::ATTN_CLUSTER - 1) / bq::ATTN_CLUSTER + 63) / 64 * 64;
    if (n < CHUNK_MIN) n = CHUNK_MIN;
    const int64_t units = pairs * ((capacity + n - 1) / n);
    if (n <= CLUSTER_CHUNK && units <= TARGET) return {(int)n, capacity > n};
    n = ((pairs * capacity + TARGET - 1) / TARGET + 63) / 64 * 64;
    n = n < CHUNK_MIN ? CHUNK_MIN : n > CHUNK_MAX ? CHUNK_MAX : n;
    return {(int)n, false};
}

// validation of shapes and choice of the instance
bq_status plan_of(const bq_kv_cache *c, const bq_attention_args *x, Plan *p, bool shared = false) {
    if (!c || !x) return BQ_ERR_NULL;
    const bq_status s = bq::check_attention_shape(c, x);
    if (s != BQ_OK) return s;
    bq::AttnArgs &a = p->a;
    a.c = *c;
    a.x = *x;
    a.page.set((uint32_t)c->page_size);
    a.group.set((uint32_t)(x->heads / c->kv_heads));
    a.group_rows = x->heads / c->kv_heads * x->rows;
    const int64_t capacity = (int64_t)x->table_width * c->page_size;
    const Chunking how = chunking_of(x->requests, c->kv_heads, capacity);
    a.chunk = how.chunk;
    a.cluster = how.cluster;
    a.max_chunks = bq::attn_chunks((int)capacity, a.chunk);
    a.scale_log2 = x->scale * 1.44269504088896340736f;
    a.mode = bq::ATTN_ALL;
    const int nt = bq::attn_tiles(c, a.group_rows);
    a.row_tiles = (a.group_rows + 8 * nt - 1) / (8 * nt);
    p->inst = bq::attn_instance(c, x->dtype, nt, shared);
    if (!p->inst) return BQ_ERR_SHAPE;
    p->smem = p->inst->smem + (size_t)(x->requests + 1) * sizeof(int);
    p->units = (int64_t)x->requests * a.max_chunks * c->kv_heads * a.row_tiles;
    if ((int64_t)x->requests * a.max_chunks > 0x7fffffffLL || p->units > (1LL << 40) ||
        (int64_t)x->requests * x->rows * x->heads > 0x7fffffffLL)
        return BQ_ERR_SHAPE;
    const int64_t rows = a.max_chunks > 1 && !a.cluster ? p->units * 8 * nt : 0;
    p->ml_bytes = (rows * (int64_t)sizeof(float2) + 15) / 16 * 16;
    p->o_bytes = rows * c->head_dim * (int64_t)sizeof(float);
    return BQ_OK;
}

}  // namespace

namespace bq {

bq_status check_attention_shape(const bq_kv_cache *c, const bq_attention_args *x) {
    const bq_status s = check_cache_shape(c);
    if (s != BQ_OK) return s;
    if (!dtype_bytes(x->dtype)) return BQ_ERR_QTYPE;
    if (x->requests < 0 || x->requests > ATTN_MAX_REQUESTS || x->rows < 1 || x->rows > BQ_VERIFY_MAX_ROWS ||
        x->heads < 1 || x->heads > 4096 || x->heads % c->kv_heads || x->table_width < 1 ||
        (int64_t)x->table_width * c->page_size > (1LL << 23) || x->table_stride < x->table_width ||
        x->table_stride > (1LL << 40) || !std::isfinite(x->scale))
        return BQ_ERR_SHAPE;
    const int64_t strides[] = {x->q_row_stride, x->q_head_stride, x->out_row_stride, x->out_head_stride};
    for (int64_t v : strides)
        if (v < 0 || v > (1LL << 40)) return BQ_ERR_SHAPE;
    return BQ_OK;
}

bq_status check_attention_pointers(const bq_kv_cache *c, const bq_attention_args *x) {
    const bq_status s = check_cache_pointers(c);
    if (s != BQ_OK) return s;
    if (!x->q || !x->out || !x->table || !x->lens) return BQ_ERR_NULL;
    const uintptr_t es = (uintptr_t)dtype_bytes(x->dtype);
    if (!aligned_to(x->q, es) || !aligned_to(x->out, es) || !aligned_to(x->table, 4) || !aligned_to(x->lens, 4))
        return BQ_ERR_ALIGN;
    return BQ_OK;
}

static int padded_dim(const bq_kv_cache *c) { return c->head_dim <= 64 ? 64 : c->head_dim <= 128 ? 128 : 256; }

// 8 query rows per n-tile, as few row tiles as the registers allow: each
// reads the cache again.  A Q8_0 cache takes two n-tiles at most: with four its
// code outgrows the instruction cache (5 rows of 40 heads over 8, 24577
// positions: 57 us against 63).
int attn_tiles(const bq_kv_cache *c, int64_t group_rows) {
    return group_rows <= 8 ? 1 : group_rows <= 16 || padded_dim(c) == 256 || c->type == BQ_Q8_0 ? 2 : 4;
}

const AttnInstance *attn_instance(const bq_kv_cache *c, int dtype, int nt, bool modes) {
    using Table = const AttnInstance *(*)(int *);
    const bool same = dtype == c->type;
    const Table of[3][2][2] = {
        {{bq_internal_attn_f16_split, bq_internal_attn_f16_own},
         {bq_internal_attn_f16_split_shared, bq_internal_attn_f16_own_shared}},
        {{bq_internal_attn_bf16_split, bq_internal_attn_bf16_own},
         {bq_internal_attn_bf16_split_shared, bq_internal_attn_bf16_own_shared}},
        {{bq_internal_attn_q8_0_split, bq_internal_attn_q8_0_own},
         {bq_internal_attn_q8_0_split_shared, bq_internal_attn_q8_0_own_shared}}};
    const int kind = c->type == BQ_F16 ? 0 : c->type == BQ_BF16 ? 1 : 2;
    int n = 0;
    const AttnInstance *inst = of[kind][modes][kind == 2 ? dtype != BQ_F32 : same](&n);
    for (int i = 0; i < n; ++i)
        if (inst[i].dim == padded_dim(c) && inst[i].nt == nt) return &inst[i];
    return nullptr;
}

}  // namespace bq

int bq_internal_status_attn(unsigned int *flags, int clear) {
    unsigned int a = 0, b = 0;
    int e = read_status_attn(&a, clear);
    if (e == 0) e = bq_internal_status_attn_prefix(&b, clear);
    *flags = a | b;
    return e;
}

// host hooks for the tests (not in the public header): the launch constant's
// quotient, and how a call is cut: chunk, chunks, cluster, row tiles
extern "C" unsigned int bq_internal_fast_div(unsigned int n, unsigned int d) {
    bq::FastDiv f;
    f.set(d);
    return f.div(n);
}
extern "C" int bq_internal_attention_plan(const bq_kv_cache *cache, const bq_attention_args *args, int *out) {
    Plan p;
    const bq_status s = plan_of(cache, args, &p);
    if (s == BQ_OK) out[0] = p.a.chunk, out[1] = p.a.max_chunks, out[2] = p.a.cluster, out[3] = p.a.row_tiles;
    return (int)s;
}

extern "C" int64_t bq_paged_attention_workspace_bytes(const bq_kv_cache *cache, const bq_attention_args *args) {
    Plan p;
    if (plan_of(cache, args, &p) != BQ_OK) return -1;
    return p.ml_bytes + p.o_bytes;
}

// the call, over the groups of `shared` if there are any
bq_status bq_internal_paged_attention(const bq_kv_cache *cache, const bq_attention_args *x, const bq::AttnArgs *shared,
                                      void *workspace, int64_t workspace_bytes, void *stream) {
    Plan p;
    bq_status s = plan_of(cache, x, &p, shared != nullptr);
    if (s != BQ_OK) return s;
    if (x->requests == 0) return BQ_OK;
    s = bq::check_attention_pointers(cache, x);
    if (s != BQ_OK) return s;
    bq::AttnArgs &a = p.a;
    if (shared) {
        a.mode = bq::ATTN_WHOLE;
        for (int g = 0; g < bq::ATTN_GROUPS; ++g)
            a.group_end[g] = shared->group_end[g], a.group_pages[g] = shared->group_pages[g];
    }
    const int64_t need = p.ml_bytes + p.o_bytes;
    if (need) {
        if (!workspace) return BQ_ERR_NULL;
        if (!bq::aligned_to(workspace, 16)) return BQ_ERR_ALIGN;
        if (workspace_bytes < need) return BQ_ERR_SHAPE;
    }
    a.part_ml = static_cast<float2 *>(workspace);
    a.part_o = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + p.ml_bytes);
    const int sms = bq::device_sms();
    if (!sms) return BQ_ERR_CUDA;
    int occ = 0;
    if (p.inst->occupancy(p.smem, &occ) != 0 || occ < 1) return bq::from_cuda_error(cudaErrorInvalidConfiguration);
    const int64_t slots = (int64_t)sms * occ;
    // Up to DIRECT units per slot the hardware hands them out as CTAs end, whole
    // chunks before ragged ones (48 requests to 12001: 202 us against 210; Q8_0, 48 to
    // 6000, bf16 queries: 92 against 107).  A unit behind its request's length costs about 4 ns of the
    // GPU then, so a table much wider than the requests goes by the scan of the
    // lengths instead.
    constexpr int64_t DIRECT = 8;
    a.direct = a.cluster || p.units <= DIRECT * slots;
    if (a.cluster && p.units > 0x7fffffffLL) return BQ_ERR_SHAPE;
    const int64_t grid = a.direct || p.units < slots ? p.units : slots;
    unsigned int *status = nullptr;
    cudaError_t e = status_address(&status);
    if (e == cudaSuccess) e = p.inst->launch(a, (int)grid, p.smem, stream, status);
    if (e != cudaSuccess || a.max_chunks == 1 || a.cluster) return bq::from_cuda_error(e);
    const int tile_rows = 8 * p.inst->nt;
    e = x->dtype == BQ_F32   ? join<BQ_F32>(a, tile_rows, stream)
        : x->dtype == BQ_F16 ? join<BQ_F16>(a, tile_rows, stream)
                             : join<BQ_BF16>(a, tile_rows, stream);
    return bq::from_cuda_error(e);
}

extern "C" bq_status bq_paged_attention(const bq_kv_cache *cache, const bq_attention_args *x, void *workspace,
                                        int64_t workspace_bytes, void *stream) {
    return bq_internal_paged_attention(cache, x, nullptr, workspace, workspace_bytes, stream);
}
