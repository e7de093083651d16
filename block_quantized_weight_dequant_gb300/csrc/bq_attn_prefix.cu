// bq_attn_prefix.cu -- attention of requests that share the first pages of their
// histories (bq_paged_prefix_attention in include/bqgemv.h): planning and join.
//
// Mathematics.  A row's positions are the shared ones and those behind them; with
// the partial maximum m, sum l and unnormalised O of any cut of them
//   o = sum_i 2^(m_i - max m) O_i / sum_i 2^(m_i - max m) l_i.
// So the shared pages are gone through once for all query rows of a group of
// requests (rows of one kv head side by side), the rest once per request by the
// kernel that serves ordinary calls, and the partial results of both are joined
// here, in a fixed order: a row's bits depend on its own inputs and the call's
// geometry alone.
//
// Bounds: by size, the shared pass (96 requests of 32801 shared, bf16, 32 over 8 heads of
// 128: 125 us a call, 96 of them that pass), the ordinary kernel's instructions (16
// requests of 30011 over Q8_0: 58 us) or the chain of three launches (200 requests in 3
// groups of 9001: 31 us).
// The launches follow one another, each waiting for the one before to end: own pages that
// started while the shared ones were gone through, without that wait, took 8, 5 and 1 us
// less, but nothing that is documented orders their reads behind the writes before the call.
#include <atomic>
#include <cmath>

#include "bq_attn_tcgen05.cuh"

// bq_attn_tcgen05_<cache>.cu
cudaError_t bq_internal_prefix_f16(const bq::TcArgs &, int grid, void *stream, unsigned int *status);
cudaError_t bq_internal_prefix_bf16(const bq::TcArgs &, int grid, void *stream, unsigned int *status);
cudaError_t bq_internal_prefix_q8_0(const bq::TcArgs &, int grid, void *stream, unsigned int *status);

namespace {

BQ_STATUS_WORD(attn_prefix)

cudaError_t status_address(unsigned int **out) {
    static std::atomic<unsigned int *> addr[64];
    return bq::symbol_address(addr, g_status_attn_prefix, out);
}

constexpr int JOIN_THREADS = 256;

// partial results of one of the two passes
struct Parts {
    const float *o;
    const float2 *ml;
    int chunk, max_chunks, row_tiles, tile_rows;
};
struct JoinArgs {
    bq::AttnArgs a;  // of the rest
    Parts shared, rest;
};

// W warps per query row and head: warp w takes the partial results w, w + W, ...
// in order, then the warps' sums are added in order.
template <int DT, int W, int DB>
__global__ void __launch_bounds__(JOIN_THREADS, 4) prefix_join_kernel(const __grid_constant__ JoinArgs j) {
    constexpr int ROWS = JOIN_THREADS / 32 / W;
    __shared__ float4 o_s[W > 1 ? W : 1][W > 1 ? 32 * DB : 1];
    __shared__ float2 ml_s[W];
    const bq::AttnArgs &a = j.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, w = W > 1 ? warp : 0;
    const int D = a.c.head_dim, R = a.x.rows, KVH = a.c.kv_heads, G = (int)a.group.d;
    const int index = (int)blockIdx.x * ROWS + (W > 1 ? 0 : warp);  // (rows and heads are below 2^27)
    bq::pdl_wait();
    const int token = index / a.x.heads, head = index - token * a.x.heads;
    const int b = token / R, row = token - b * R;
    if (b >= a.x.requests) return;  // (W > 1: there is no such row)
    const int h = head / G, in_group = head - h * G;
    int g = 0;
    while (a.group_end[g] <= b) ++g;
    const int first = g ? a.group_end[g - 1] : 0;
    const int common = a.group_pages[g] * a.c.page_size;
    const int len = bq::attn_clamped(a.x.lens[b], a.x.table_width * a.c.page_size);
    const bool sees = bq::attn_sees(len, R, common);  // else neither pass has anything for it
    const int ns = sees && common ? bq::attn_chunks(common, j.shared.chunk) : 0;
    const int n = ns + (sees ? bq::attn_chunks(bq::attn_rest(len, R, common), j.rest.chunk) : 0);
    const int si = ((b - first) * R + row) * G + in_group, ri = row * G + in_group;
    // where the partial results of each pass lie, in rows: the first and the distance
    auto first_of = [&](const Parts &p, int of, int i) {
        const int t = i / p.tile_rows;
        return (((long long)of * p.max_chunks * KVH + h) * p.row_tiles + t) * p.tile_rows + (i - t * p.tile_rows);
    };
    const long long s0 = first_of(j.shared, g, si), sn = (long long)KVH * j.shared.row_tiles * j.shared.tile_rows;
    const long long r0 = first_of(j.rest, b, ri), rn = (long long)KVH * j.rest.row_tiles * j.rest.tile_rows;
    const float *s_o = j.shared.o + s0 * D + 4 * lane, *r_o = j.rest.o + r0 * D + 4 * lane;
    const long long s_hop = sn * D, r_hop = rn * D;
    auto stats = [&](int k) { return k < ns ? j.shared.ml[s0 + k * sn] : j.rest.ml[r0 + (k - ns) * rn]; };
    // AHEAD partial results are on their way while the weights of up to 32 are found;
    // with more, those come 32 at a time, with a running maximum
    constexpr int AHEAD = 4;
    float top = -INFINITY, sum = 0.0f;
    float4 acc[DB] = {};
    auto fetch = [&](int k, float4(&v)[DB]) {
        const float *src = k < ns ? s_o + k * s_hop : r_o + (k - ns) * r_hop;
#pragma unroll
        for (int e = 0; e < DB; ++e)
            if (128 * e + 4 * lane < D) v[e] = *reinterpret_cast<const float4 *>(src + 128 * e);
    };
    for (int k0 = w; k0 < n; k0 += W * 32) {
        const int mine = k0 + W * lane, many = min(32, (n - k0 + W - 1) / W);
        const float2 ml = mine < n ? stats(mine) : make_float2(-INFINITY, 0.0f);
        float4 o[AHEAD][DB];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            if (i < many) fetch(k0 + W * i, o[i]);
        float now = ml.x;
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) now = fmaxf(now, __shfl_xor_sync(~0u, now, s));
        now = fmaxf(now, top);
        const float back = top == -INFINITY ? 0.0f : exp2f(top - now);
        top = now;
        const float f = ml.x == -INFINITY ? 0.0f : exp2f(ml.x - top);
        float part = f * ml.y;
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) part += __shfl_xor_sync(~0u, part, s);
        sum = fmaf(sum, back, part);
        if (k0 > w) {
#pragma unroll
            for (int e = 0; e < DB; ++e) acc[e].x *= back, acc[e].y *= back, acc[e].z *= back, acc[e].w *= back;
        }
        for (int i0 = 0; i0 < many; i0 += AHEAD) {
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                if (i0 + i >= many) break;
                const float x = __shfl_sync(~0u, f, i0 + i);
#pragma unroll
                for (int e = 0; e < DB; ++e) {
                    acc[e].x = fmaf(x, o[i][e].x, acc[e].x);
                    acc[e].y = fmaf(x, o[i][e].y, acc[e].y);
                    acc[e].z = fmaf(x, o[i][e].z, acc[e].z);
                    acc[e].w = fmaf(x, o[i][e].w, acc[e].w);
                }
            }
#pragma unroll
            for (int i = 0; i < AHEAD; ++i)
                if (i0 + AHEAD + i < many) fetch(k0 + W * (i0 + AHEAD + i), o[i]);
        }
    }
    if constexpr (W > 1) {
        if (lane == 0) ml_s[w] = make_float2(top, sum);
#pragma unroll
        for (int e = 0; e < DB; ++e) o_s[w][lane + 32 * e] = acc[e];
        __syncthreads();
        if (w) return;
        top = -INFINITY;
        for (int i = 0; i < W; ++i) top = fmaxf(top, ml_s[i].x);
        sum = 0.0f;
#pragma unroll
        for (int e = 0; e < DB; ++e) acc[e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int i = 0; i < W; ++i) {
            const float x = ml_s[i].x == -INFINITY ? 0.0f : exp2f(ml_s[i].x - top);
            sum = fmaf(x, ml_s[i].y, sum);
#pragma unroll
            for (int e = 0; e < DB; ++e) {
                const float4 v = o_s[i][lane + 32 * e];
                acc[e].x = fmaf(x, v.x, acc[e].x);
                acc[e].y = fmaf(x, v.y, acc[e].y);
                acc[e].z = fmaf(x, v.z, acc[e].z);
                acc[e].w = fmaf(x, v.w, acc[e].w);
            }
        }
    }
    const long long to = (long long)token * a.x.out_row_stride + (long long)head * a.x.out_head_stride;
#pragma unroll
    for (int e = 0; e < DB; ++e) {
        const int d = 128 * e + 4 * lane;
        if (d >= D) break;
        const float v[4] = {acc[e].x, acc[e].y, acc[e].z, acc[e].w};
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const float y = sum == 0.0f ? 0.0f : v[x] / sum;  // a row that sees nothing
            if constexpr (DT == BQ_F32) ((float *)a.x.out)[to + d + x] = y;
            else if constexpr (DT == BQ_F16) ((__half *)a.x.out)[to + d + x] = __float2half_rn(y);
            else ((__nv_bfloat16 *)a.x.out)[to + d + x] = __float2bfloat16_rn(y);
        }
    }
}

template <int DT, int W>
cudaError_t join(const JoinArgs &j, int64_t rows, void *stream) {
    constexpr int PER = JOIN_THREADS / 32 / W;
    auto *kern = j.a.c.head_dim <= 128 ? prefix_join_kernel<DT, W, 1> : prefix_join_kernel<DT, W, 2>;
    return bq::launch_pdl(kern, dim3((unsigned)((rows + PER - 1) / PER)), JOIN_THREADS, 0, stream, 1, j);
}
template <int DT>
cudaError_t join(const JoinArgs &j, void *stream) {
    const int64_t rows = (int64_t)j.a.x.requests * j.a.x.rows * j.a.x.heads;
    // a warp per row where there are rows enough and few partial results of each
    return rows >= 2048 && j.shared.max_chunks + j.rest.max_chunks <= 32 ? join<DT, 1>(j, rows, stream)
                                                                         : join<DT, 8>(j, rows, stream);
}

// one pass of the attention kernel: its arguments, instance and partial results
struct Pass {
    bq::AttnArgs a;
    const bq::AttnInstance *inst;  // NULL: the tensor-memory kernel
    int tile_rows;
    int64_t units, ml_bytes, o_bytes;
};
struct Plan {
    Pass rest, shared;
    bool any_shared;
    bool whole;     // one pass of the ordinary kernel instead
    int64_t bytes;  // of workspace
};

// Positions per unit: about TARGET units (two CTAs on each of 152 SMs), 128 at
// least, 2048 at most.
constexpr int64_t TARGET = 304, CHUNK_MIN = 128, CHUNK_MAX = 2048;
int chunk_of(int64_t pairs, int64_t positions) {
    const int64_t n = ((pairs * positions + TARGET - 1) / TARGET + 63) / 64 * 64;
    return (int)(n < CHUNK_MIN ? CHUNK_MIN : n > CHUNK_MAX ? CHUNK_MAX : n);
}

bool size_parts(Pass *p, int requests) {
    const bq_kv_cache *c = &p->a.c;
    p->a.cluster = 0;
    p->units = (int64_t)requests * p->a.max_chunks * c->kv_heads * p->a.row_tiles;
    if ((int64_t)requests * p->a.max_chunks > 0x7fffffffLL || p->units > (1LL << 40)) return false;
    const int64_t part_rows = p->units * p->tile_rows;
    p->ml_bytes = (part_rows * (int64_t)sizeof(float2) + 15) / 16 * 16;
    p->o_bytes = part_rows * c->head_dim * (int64_t)sizeof(float);
    return true;
}

bool size_pass(Pass *p, int requests, int64_t rows, int64_t positions, int pairs_of) {
    const bq_kv_cache *c = &p->a.c;
    const int nt = bq::attn_tiles(c, rows);
    p->inst = bq::attn_instance(c, p->a.x.dtype, nt, true);
    if (!p->inst) return false;
    p->tile_rows = 8 * nt;
    p->a.group_rows = (int)rows;
    p->a.row_tiles = (int)((rows + 8 * nt - 1) / (8 * nt));
    p->a.chunk = chunk_of((int64_t)pairs_of * c->kv_heads * p->a.row_tiles, positions);
    p->a.max_chunks = bq::attn_chunks((int)positions, p->a.chunk);
    return size_parts(p, requests);
}

// The tensor-memory kernel for heads of up to 128 values: tiles of 128 rows, chunks
// of whole tiles of positions, one CTA per SM.  Over a Q8_0 cache, whose codes it has
// to put into two 16-bit parts, for more rows of a kv head than two passes of the
// ordinary kernel's 16: 30011 shared, 8 kv heads of 128, fp32 queries, 32 rows 65 us
// against 57, 48 rows 74 against 92, 128 rows 92 against 189.
constexpr int64_t Q8_ROWS = 32;
bool has_tensor_kernel(const bq_kv_cache *c, int64_t rows) {
    return c->head_dim <= 128 && (c->type != BQ_Q8_0 || rows > Q8_ROWS);
}
constexpr int TILE_ROWS = 128;
// positions of its tiles, as TcShape has them
int tile_positions(const bq_kv_cache *c) { return c->type == BQ_F16 ? 128 : 64; }

// Tiles of a chunk: the fewest steps of the whole GPU, a chunk's start, joins and
// partial results counted as FIXED tiles.  At most 8192 positions, or 4096 of a Q8_0
// cache, whose parts go by the chunk's largest scale.
bool size_tensor_pass(Pass *p, int groups, int64_t rows, int64_t positions, int sms) {
    constexpr int FIXED = 6;
    const int TILE = tile_positions(&p->a.c), MOST = (p->a.c.type == BQ_Q8_0 ? 4096 : 8192) / TILE;
    p->inst = nullptr;
    p->tile_rows = TILE_ROWS;
    p->a.group_rows = (int)rows;
    p->a.row_tiles = (int)((rows + TILE_ROWS - 1) / TILE_ROWS);
    const int64_t pairs = (int64_t)p->a.c.kv_heads * p->a.row_tiles;
    const int64_t tiles = (positions + TILE - 1) / TILE;
    auto units_of = [&](int64_t n) {  // with n tiles a chunk
        int64_t units = 0;
        for (int g = 0; g < groups; ++g) {
            const int64_t of = (int64_t)p->a.group_pages[g] * p->a.c.page_size;
            const int64_t requests = p->a.group_end[g] - (g ? p->a.group_end[g - 1] : 0);
            const int64_t row_tiles = (requests * p->a.x.rows * (int)p->a.group.d + TILE_ROWS - 1) / TILE_ROWS;
            units += p->a.c.kv_heads * row_tiles * ((of + n * TILE - 1) / (n * TILE));
        }
        return units;
    };
    const int64_t most = tiles < MOST ? tiles : MOST;
    int64_t best = 0, cost = 0;
    for (int64_t steps = 1; steps <= 4; ++steps) {  // the smallest chunk that gives so many steps
        int64_t lo = 1, hi = most;
        while (lo < hi) {
            const int64_t mid = (lo + hi) / 2;
            if (units_of(mid) <= steps * sms) hi = mid;
            else lo = mid + 1;
        }
        const int64_t now = (units_of(lo) + sms - 1) / sms * (lo + FIXED);
        if (!best || now < cost) best = lo, cost = now;
    }
    p->a.chunk = (int)best * TILE;
    p->a.max_chunks = bq::attn_chunks((int)positions, p->a.chunk);
    if ((int64_t)groups * pairs * p->a.max_chunks > 0x7fffffffLL) return false;
    return size_parts(p, groups);
}

// Shared keys and values, counted once for each request of a group but one (a group of
// one reads nothing again), up to which the ordinary kernel serves the call in one pass.
// Measured, the calls captured in a graph, 16 heads over 8 of 128, one pass and shared:
//                                        fp16       bf16       fp32 / fp16  fp32 / Q8_0
//    16 M values (2 requests of 8192)     13.4 18.8  13.9 22.0  14.4 26.5    15.1 16.6 us
//    30 M (16 of 1024)                    15.2 18.1  15.7 17.4  16.4 23.5    18.0 20.9
//    43 M (8 of 3136)                     19.9 17.2  20.6 17.8  21.3 22.8    21.7 20.6
//    64 M (17 of 2048)                    23.8 18.8  24.9 18.6  25.9 24.2    26.5 26.6
//   128 M (9 of 8192)                     38.2 19.8  41.0 23.1  41.8 27.4    41.6 29.6
constexpr int64_t WHOLE = 40LL << 20;
std::atomic<int64_t> whole_limit{WHOLE};

bq_status plan_of(const bq_kv_cache *c, const bq_attention_args *x, const int32_t *counts, const int32_t *shared,
                  int groups, Plan *p) {
    if (!c || !x) return BQ_ERR_NULL;
    const bq_status s = bq::check_attention_shape(c, x);
    if (s != BQ_OK) return s;
    if (groups < 1 || groups > BQ_PREFIX_MAX_GROUPS) return BQ_ERR_SHAPE;
    if (!counts || !shared) return BQ_ERR_NULL;
    const int64_t capacity = (int64_t)x->table_width * c->page_size;
    bq::AttnArgs &a = p->rest.a;
    a.c = *c;
    a.x = *x;
    a.page.set((uint32_t)c->page_size);
    a.group.set((uint32_t)(x->heads / c->kv_heads));
    a.scale_log2 = x->scale * 1.44269504088896340736f;
    int64_t end = 0, most_rest = 0, most_shared = 0, most_rows = 0;
    int sharing = 0;
    const int64_t each = (int64_t)(x->heads / c->kv_heads) * x->rows;
    for (int g = 0; g < groups; ++g) {
        if (counts[g] < 0 || shared[g] < 0 || shared[g] > capacity) return BQ_ERR_SHAPE;
        end += counts[g];
        if (end > x->requests) return BQ_ERR_SHAPE;
        const int pages = counts[g] ? shared[g] / c->page_size : 0;
        a.group_end[g] = (int)end;
        a.group_pages[g] = pages;
        const int64_t common = (int64_t)pages * c->page_size;
        if (counts[g] && capacity - common > most_rest) most_rest = capacity - common;
        if (common > most_shared) most_shared = common;
        if (common && counts[g] * each > most_rows) most_rows = counts[g] * each;
        sharing += common != 0;
    }
    if (end != x->requests) return BQ_ERR_SHAPE;
    for (int g = groups; g < bq::ATTN_GROUPS; ++g) a.group_end[g] = (int)end, a.group_pages[g] = 0;
    p->any_shared = sharing != 0;
    // What the shared pages would be read again for all requests, against the launches
    // that sharing costs (WHOLE has the figures).
    int64_t again = 0;
    for (int g = 0; g < groups; ++g)
        if (counts[g])
            again += 2LL * (counts[g] - 1) * a.group_pages[g] * c->page_size * c->kv_heads * c->head_dim;
    p->whole = !p->any_shared || again < whole_limit.load(std::memory_order_relaxed);
    if (p->whole) {
        p->bytes = bq_paged_attention_workspace_bytes(c, x);
        return p->bytes < 0 ? BQ_ERR_SHAPE : BQ_OK;
    }
    p->shared.a = a;
    a.mode = bq::ATTN_REST;
    if (!size_pass(&p->rest, x->requests, each, most_rest, x->requests)) return BQ_ERR_SHAPE;
    {
        bq::AttnArgs &b = p->shared.a;
        b.mode = bq::ATTN_PREFIX;
        b.x.requests = groups;
        // (152 SMs whatever the device: the workspace's size is told without one)
        if (has_tensor_kernel(c, most_rows) ? !size_tensor_pass(&p->shared, groups, most_rows, most_shared, 152)
                                 : !size_pass(&p->shared, groups, most_rows, most_shared, sharing))
            return BQ_ERR_SHAPE;
    }
    p->bytes = p->rest.ml_bytes + p->rest.o_bytes + p->shared.ml_bytes + p->shared.o_bytes;
    return BQ_OK;
}

// A map of the pages' 64-value blocks, swizzled as the tensor cores read them;
// false if the driver has none.
bool map_of(const bq_kv_cache &c, void *base, int box, bool heads_first, const cuuint64_t *strides, CUtensorMap *out) {
    using Encode = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static std::atomic<Encode> known{nullptr};
    Encode encode = known.load();
    if (!encode) {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess || !p) {
            cudaGetLastError();
            return false;
        }
        encode = reinterpret_cast<Encode>(p);
        known.store(encode);
    }
    const cuuint64_t dims[4] = {(cuuint64_t)c.head_dim, (cuuint64_t)(heads_first ? c.kv_heads : c.page_size),
                                (cuuint64_t)(heads_first ? c.page_size : c.kv_heads), (cuuint64_t)c.pages};
    const cuuint32_t boxes[4] = {64, (cuuint32_t)(heads_first ? 1 : box), (cuuint32_t)(heads_first ? box : 1), 1};
    const cuuint32_t steps[4] = {1, 1, 1, 1};
    return encode(out, c.type == BQ_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims,
                  strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Boxes and maps of the call's copies; box 0, the copies of 16 bytes, where pages are
// not whole groups of 8 slots or the strides are none of a tensor map's (each a
// multiple of the one before, and beyond what that spans).
void maps_of(const bq_kv_cache &c, bq::TcArgs *t) {
    const int most = tile_positions(&c);
    t->box = c.page_size & -c.page_size;  // the largest power of two that divides it
    if (t->box > most) t->box = most;
    const cuuint64_t D = 2 * (cuuint64_t)c.head_dim, S = (cuuint64_t)c.page_size, H = (cuuint64_t)c.kv_heads;
    const cuuint64_t slot = 2 * (cuuint64_t)c.slot_stride;
    const cuuint64_t head = H > 1 ? 2 * (cuuint64_t)c.head_stride : slot * S;  // (one entry has no stride)
    t->heads_first = head < slot;
    const cuuint64_t n0 = t->heads_first ? H : S, n1 = t->heads_first ? S : H;
    cuuint64_t strides[3] = {t->heads_first ? head : slot, t->heads_first ? slot : head, 0};
    strides[2] = c.pages > 1 ? 2 * (cuuint64_t)c.page_stride : strides[1] * n1;
    const bool fits = t->box >= 8 && strides[0] >= D && strides[1] >= strides[0] * n0 && strides[1] % strides[0] == 0 &&
                      strides[2] >= strides[1] * n1 && strides[2] % strides[1] == 0;
    if (!fits || !map_of(c, c.k, t->box, t->heads_first, strides, &t->k) ||
        !map_of(c, c.v, t->box, t->heads_first, strides, &t->v))
        t->box = 0;
}

// waits of the tensor-memory kernel: their limit, and a barrier to hold (for the tests)
constexpr uint64_t WAIT_NS = 1000000000;
std::atomic<uint64_t> wait_ns{WAIT_NS};
std::atomic<int> hold{bq::TC_HOLD_NONE};

cudaError_t run(Pass *p, int sms, void *stream, unsigned int *status) {
    if (!p->inst) {
        bq::TcArgs t;
        t.a = p->a;
        const bq_kv_cache &c = p->a.c;
        t.box = t.heads_first = 0;
        t.wait_ns = wait_ns.load(std::memory_order_relaxed);
        t.hold = hold.load(std::memory_order_relaxed);
        if (c.type == BQ_Q8_0) return bq_internal_prefix_q8_0(t, (int)p->units, stream, status);
        maps_of(c, &t);
        return c.type == BQ_F16 ? bq_internal_prefix_f16(t, (int)p->units, stream, status)
                                : bq_internal_prefix_bf16(t, (int)p->units, stream, status);
    }
    const size_t smem = p->inst->smem + (size_t)(p->a.x.requests + 1) * sizeof(int);
    int occ = 0;
    if (p->inst->occupancy(smem, &occ) != 0 || occ < 1) return cudaErrorInvalidConfiguration;
    const int64_t slots = (int64_t)sms * occ;
    constexpr int64_t DIRECT = 8;  // as in bq_paged_attention
    p->a.direct = p->units <= DIRECT * slots;
    const int64_t grid = p->a.direct || p->units < slots ? p->units : slots;
    return p->inst->launch(p->a, (int)grid, smem, stream, status);
}

Parts parts_of(const Pass &p) {
    return {p.a.part_o, p.a.part_ml, p.a.chunk, p.a.max_chunks, p.a.row_tiles, p.tile_rows};
}

}  // namespace

int bq_internal_status_attn_prefix(unsigned int *flags, int clear) { return read_status_attn_prefix(flags, clear); }

// host hook for the tests (not in the public header): sets the limit, returns the one before
extern "C" int64_t bq_internal_prefix_whole_limit(int64_t bytes) { return whole_limit.exchange(bytes < 0 ? WHOLE : bytes); }

// likewise: calls from now on hold a barrier (a TcHold, 0: none) and wait for wait_ns at
// most (0: the ordinary limit); nonzero for a barrier that there is not
extern "C" int bq_internal_prefix_hold(int barrier, unsigned long long limit_ns) {
    if (barrier < 0 || barrier >= bq::TC_HOLD_KINDS) return -1;
    hold.store(barrier);
    wait_ns.store(limit_ns ? limit_ns : WAIT_NS);
    return 0;
}

extern "C" int64_t bq_paged_prefix_attention_workspace_bytes(const bq_kv_cache *cache, const bq_attention_args *args,
                                                             const int32_t *group_requests, const int32_t *group_shared,
                                                             int groups) {
    Plan p;
    return plan_of(cache, args, group_requests, group_shared, groups, &p) == BQ_OK ? p.bytes : -1;
}

extern "C" bq_status bq_paged_prefix_attention(const bq_kv_cache *cache, const bq_attention_args *x,
                                               const int32_t *group_requests, const int32_t *group_shared, int groups,
                                               void *workspace, int64_t workspace_bytes, void *stream) {
    Plan p;
    bq_status s = plan_of(cache, x, group_requests, group_shared, groups, &p);
    if (s != BQ_OK) return s;
    if (x->requests == 0) return BQ_OK;
    s = bq::check_attention_pointers(cache, x);
    if (s != BQ_OK) return s;
    if (p.whole) return bq_internal_paged_attention(cache, x, &p.rest.a, workspace, workspace_bytes, stream);
    if (!workspace) return BQ_ERR_NULL;
    if (!bq::aligned_to(workspace, 16)) return BQ_ERR_ALIGN;
    if (workspace_bytes < p.bytes) return BQ_ERR_SHAPE;
    uint8_t *at = static_cast<uint8_t *>(workspace);
    for (Pass *pass : {&p.rest, &p.shared}) {
        pass->a.part_ml = reinterpret_cast<float2 *>(at);
        pass->a.part_o = reinterpret_cast<float *>(at + pass->ml_bytes);
        at += pass->ml_bytes + pass->o_bytes;
    }
    const int sms = bq::device_sms();
    if (!sms) return BQ_ERR_CUDA;
    unsigned int *status = nullptr;
    cudaError_t e = status_address(&status);
    if (e == cudaSuccess) e = run(&p.shared, sms, stream, status);
    if (e == cudaSuccess) e = run(&p.rest, sms, stream, status);
    if (e != cudaSuccess) return bq::from_cuda_error(e);
    JoinArgs j;
    j.a = p.rest.a;
    j.rest = parts_of(p.rest);
    j.shared = parts_of(p.shared);
    e = x->dtype == BQ_F32   ? join<BQ_F32>(j, stream)
        : x->dtype == BQ_F16 ? join<BQ_F16>(j, stream)
                             : join<BQ_BF16>(j, stream);
    return bq::from_cuda_error(e);
}
