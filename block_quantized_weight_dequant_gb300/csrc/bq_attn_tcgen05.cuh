// bq_attn_tcgen05.cuh -- the shared pages of a group of requests gone through once
// for all its query rows (the first pass of bq_paged_prefix_attention in
// include/bqgemv.h) over 16-bit caches with heads of up to 128 values.
//
// Mathematics.  For 128 query rows of one kv head at a time and tiles of 128
// positions: S = Q K^T, P = 2^(factor S - m), O = O + P V with a running reference
// m and sum l per row.  m follows the running maximum only when that has grown
// by more than 2^8: weights are at most 2^8 then and O, which stays in tensor
// memory, is rescaled (by the row's own 2^(m_old - m)) in few tiles.
//
// A CTA takes a chunk of the positions for 128 rows.  Warps 0 to 3 and 4 to 7 are
// two streams: they take the even and the odd tiles, each with S (128 columns of
// tensor memory) and O (up to 128) of its own, so that the tensor cores work for
// one stream while the other one computes its weights; their O are joined at the
// end.  Warps 8 to 11 bring K and V tiles into a ring in shared memory by 16-byte
// asynchronous copies (any page size and stride; what is not there is filled with
// zeros) in the swizzled rows of 128 bytes that the tensor cores read: K with
// positions as rows and head_dim contiguous, V the same bytes with the summed
// axis as rows.  One thread of warp 12 issues all products.  The weights go back
// to tensor memory in the columns of the scores that they come from, and are the
// first operand of the second product from there.
//
// Precision.  A query of the cache's type is used as it is, any other in QP 16-bit
// parts (fp16 2, after scaling the row by a power of two; bf16 3); weights are two
// parts: 22 bits over an fp16 cache, 16 over bf16, where a third would not fit
// beside S in tensor memory (an output's error from it is below 2^-17 of the mean
// |v|; one part alone would leave 2^-9).  O sums a chunk's tiles in the tensor
// core's fp32.
#pragma once

#include <atomic>
#include <cmath>

#include "bq_attn.h"

namespace bq {

constexpr int TC_ROWS = 128, TC_TILE = 128;
constexpr int TC_SOFTMAX_WARPS = 8, TC_COPY_WARPS = 4, TC_WARPS = 13;
constexpr int TC_MASKS = 8;        // tiles whose masks are kept
constexpr int TC_BLOCK = 128 * 128;  // bytes of 128 rows of 64 values
constexpr int TC_COLUMNS = 512;      // of tensor memory, all of it
constexpr float TC_GROWTH = 8.0f;    // log2 of what a weight may be
constexpr int TC_SHIFT_F16 = 7;      // fp16 weights carry 2^7: up to 2^15, two parts keep 2^-24

template <int QP, int NB>
struct TcShape {
    static constexpr int SLOT = NB * TC_BLOCK, Q_BYTES = QP * NB * TC_BLOCK;
    static constexpr int LIMIT = 227 * 1024, MISC = 3072;
    static constexpr int most = (LIMIT - MISC - Q_BYTES) / SLOT;
    static constexpr int SLOTS = most > 8 ? 8 : most;
    // loads that are issued before the oldest is waited for.  Above SLOTS - 2 a load
    // would wait for a slot that is only freed once it has arrived.
    static constexpr int LAG = SLOTS - 3 > 4 ? 4 : SLOTS - 3;
    static constexpr int SMEM = Q_BYTES + SLOTS * SLOT + MISC;
    static constexpr int OROW = NB * 64 + 4;  // floats of a row of the join, in the ring's place
    static_assert(SLOTS >= 4 && LAG >= 1 && LAG <= SLOTS - 2);
    static_assert(TC_ROWS * OROW * 4 <= SLOTS * SLOT);
    static_assert(SMEM > 114 * 1024, "one CTA per SM: each takes all tensor memory");
    // a copying warp is at most SLOTS / 2 tiles past one whose values are in use
    static_assert(SLOTS / 2 + 1 < TC_MASKS);
};

// shared memory behind the ring
struct TcMisc {
    uint64_t full[8], empty[8], mask_full[TC_MASKS], s_full[2], p_full[2], o_full[2], q_full, last;
    uint32_t mask[TC_MASKS][4];  // positions of a tile that are there
    float factor[TC_ROWS];       // of a row's scores
    float2 ml[TC_ROWS];          // of the second stream
    uint32_t tmem;
    uint32_t dead;  // a wait has run out
};
static_assert(sizeof(TcMisc) <= 3072);

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_load() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_async_proxy() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ uint32_t tc_shared(const void *p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

__device__ __forceinline__ void barrier_init(uint64_t *b, int count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(tc_shared(b)), "r"(count) : "memory");
}
__device__ __forceinline__ void barrier_arrive(uint64_t *b) {
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(tc_shared(b)) : "memory");
}
__device__ __forceinline__ bool barrier_try(uint64_t *b, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(tc_shared(b)), "r"(parity)
        : "memory");
    return ok;
}
__device__ __forceinline__ uint64_t tc_nanoseconds() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
// Waits for a phase of the barrier, for a second at most; false if that has run
// out here or in another thread of the CTA, which then leaves its loop.
static __device__ __noinline__ bool barrier_wait_long(uint64_t *b, uint32_t parity, volatile uint32_t *dead) {
    const uint64_t t0 = tc_nanoseconds();
    while (!barrier_try(b, parity)) {
        if (*dead) return false;
        if (tc_nanoseconds() - t0 > 1000000000ull) {
            *dead = 1;
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ bool barrier_wait(uint64_t *b, uint32_t parity, volatile uint32_t *dead) {
    if (barrier_try(b, parity)) return true;
    return barrier_wait_long(b, parity, dead);
}

// 32 columns of the warp's 32 lanes of tensor memory
#define BQ_TC_32(X, v)                                                                                       \
    X(v[0]), X(v[1]), X(v[2]), X(v[3]), X(v[4]), X(v[5]), X(v[6]), X(v[7]), X(v[8]), X(v[9]), X(v[10]),      \
        X(v[11]), X(v[12]), X(v[13]), X(v[14]), X(v[15]), X(v[16]), X(v[17]), X(v[18]), X(v[19]), X(v[20]),  \
        X(v[21]), X(v[22]), X(v[23]), X(v[24]), X(v[25]), X(v[26]), X(v[27]), X(v[28]), X(v[29]), X(v[30]),  \
        X(v[31])
#define BQ_TC_OUT(x) "=r"(x)
#define BQ_TC_IN(x) "r"(x)
__device__ __forceinline__ void tc_load32(uint32_t at, uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,"
        "%28,%29,%30,%31}, [%32];"
        : BQ_TC_32(BQ_TC_OUT, v)
        : "r"(at)
        : "memory");
}
__device__ __forceinline__ void tc_store32(uint32_t at, const uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,"
        "%28,%29,%30,%31};" ::BQ_TC_32(BQ_TC_IN, v),
        "r"(at)
        : "memory");
}

// A matrix in shared memory in rows of 128 bytes swizzled over 8 rows: its place,
// the distance of 64-value blocks (where the rows are the summed axis) and of
// groups of 8 rows
__device__ __forceinline__ uint64_t tc_matrix(uint32_t at) {
    return (uint64_t)(at >> 4 & 0x3fff) | (uint64_t)(TC_BLOCK >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 |
           (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
__device__ __forceinline__ void tc_product_shared(uint32_t d, uint64_t a, uint64_t b, uint32_t shape, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(shape), "r"((uint32_t)add)
        : "memory");
}
__device__ __forceinline__ void tc_product_tensor(uint32_t d, uint32_t a, uint64_t b, uint32_t shape, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(shape), "r"((uint32_t)add)
        : "memory");
}
// the barrier's phase completes with all products issued so far
__device__ __forceinline__ void tc_commit(uint64_t *b) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(tc_shared(b))
                 : "memory");
}

__device__ __forceinline__ void tc_copy16(uint32_t dst, const void *src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
template <int N>
__device__ __forceinline__ void tc_copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ float tc_pow2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// two values as a pair of 16-bit numbers, and what is left of them
template <bool HALF>
__device__ __forceinline__ uint32_t tc_part(float &x, float &y) {
    uint32_t w;
    if constexpr (HALF) {
        w = F16::down2(x, y);
        const float2 f = F16::up2(w);
        x -= f.x, y -= f.y;
    } else {
        w = BF16::down2(x, y);
        x -= __uint_as_float(w << 16), y -= __uint_as_float(w & 0xffff0000u);
    }
    return w;
}

template <bool HALF, int QP, int NB>
__global__ void __launch_bounds__(TC_WARPS * 32, 1)
    prefix_kernel(const __grid_constant__ AttnArgs a, unsigned int *status) {
    using S = TcShape<QP, NB>;
    constexpr int SLOTS = S::SLOTS, LAG = S::LAG;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *q_s = smem, *ring = smem + S::Q_BYTES;
    TcMisc &misc = *reinterpret_cast<TcMisc *>(ring + SLOTS * S::SLOT);
    volatile uint32_t *dead = &misc.dead;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int D = a.c.head_dim, R = a.x.rows, KVH = a.c.kv_heads, G = (int)a.group.d;
    const int page = a.c.page_size;

    // ---- which rows and positions ----
    const uint32_t pairs = (uint32_t)a.x.requests * KVH * a.row_tiles;  // of the groups' tiles and kv heads
    const int ck = (int)(blockIdx.x / pairs);
    uint32_t rest = blockIdx.x - ck * pairs;
    const int rt = (int)(rest % a.row_tiles);
    rest /= a.row_tiles;
    const int h = (int)(rest % KVH), g = (int)(rest / KVH);
    const int first = g ? a.group_end[g - 1] : 0, end_request = a.group_end[g];
    const int group_rows = (end_request - first) * R * G, first_row = rt * TC_ROWS;
    const int common = a.group_pages[g] * page;
    const int begin = ck * a.chunk, end = min(begin + a.chunk, common);
    pdl_wait();
    pdl_launch_dependents();
    if (begin >= end || first_row >= group_rows) return;
    // the first request that holds the shared pages: its table row tells them
    int owner = 0x7fffffff;
    const int most = a.x.table_width * page;
    for (int i = first + lane; i < end_request && owner == 0x7fffffff; i += 32)
        if (min(a.x.lens[i], most) - R + 1 >= common) owner = i;
    owner = __reduce_min_sync(~0u, owner);
    if (owner == 0x7fffffff) return;  // nobody reads these partial results
    const int tiles = (end - begin + TC_TILE - 1) / TC_TILE;
    const int D16 = (D + 15) & ~15;

    // ---- barriers and tensor memory ----
    if (tid == 0) {
        for (int i = 0; i < SLOTS; ++i) barrier_init(&misc.full[i], TC_COPY_WARPS), barrier_init(&misc.empty[i], 1);
        for (int i = 0; i < TC_MASKS; ++i) barrier_init(&misc.mask_full[i], TC_COPY_WARPS);
        for (int i = 0; i < 2; ++i) {
            barrier_init(&misc.s_full[i], 1);
            barrier_init(&misc.p_full[i], TC_SOFTMAX_WARPS / 2);
            barrier_init(&misc.o_full[i], 1);
        }
        barrier_init(&misc.q_full, TC_SOFTMAX_WARPS);
        barrier_init(&misc.last, 1);
        misc.dead = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == TC_WARPS - 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc_shared(&misc.tmem)),
                     "n"(TC_COLUMNS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc.tmem;

    if (warp >= TC_SOFTMAX_WARPS && warp < TC_SOFTMAX_WARPS + TC_COPY_WARPS) {
        // ---- copies: K and V of each tile in turn, 32 rows of it by each warp ----
        const int cw = warp - TC_SOFTMAX_WARPS;
        const int *row_table = a.x.table + owner * a.x.table_stride;
        const long long head_off = (long long)h * a.c.head_stride;
        auto entry_of = [&](int t) { return t < end ? row_table[a.page.div((uint32_t)t)] : -1; };
        int entry = entry_of(begin + 32 * cw + lane);
        constexpr int PIECES = 8 * NB, AT_ONCE = 32 / PIECES;  // of a row; rows of a warp at a time
        const int piece = lane % PIECES, sub = lane / PIECES;
        const bool there = piece < D16 / 8, inside = 8 * piece < D;
        const uint32_t ring_at = tc_shared(ring) + (piece >> 3) * TC_BLOCK;
        auto arrived = [&](int n) {  // load n is complete: the products may read it
            fence_async_proxy();
            __syncwarp();
            if (lane == 0) barrier_arrive(&misc.full[n % SLOTS]);
        };
        bool ok = true;
        for (int t = 0; t < tiles && ok; ++t) {
            const int p = begin + t * TC_TILE + 32 * cw + lane;
            long long off = -1;
            if (p < end) {
                if (entry >= 0 && entry < a.c.pages) {
                    const uint32_t in_page = (uint32_t)p - a.page.div((uint32_t)p) * a.page.d;
                    off = entry * a.c.page_stride + in_page * a.c.slot_stride + head_off;
                } else {
                    atomicOr(status, BQ_DEVERR_PAGE);
                }
            }
            entry = entry_of(p + TC_TILE);
            const uint32_t live = __ballot_sync(~0u, off >= 0);
            for (int v = 0; v < 2; ++v) {
                const int n = 2 * t + v, slot = n % SLOTS;
                if (!barrier_wait(&misc.empty[slot], (n / SLOTS & 1) ^ 1, dead)) {
                    ok = false;
                    break;
                }
                // (after the wait: the masks of TC_MASKS tiles before are not in use any more)
                if (v == 0 && lane == 0) {
                    misc.mask[t % TC_MASKS][cw] = live;
                    barrier_arrive(&misc.mask_full[t % TC_MASKS]);
                }
                const uint8_t *src = static_cast<const uint8_t *>(v ? a.c.v : a.c.k) + 16 * piece;
                const uint32_t dst = ring_at + slot * S::SLOT;
#pragma unroll 8
                for (int i = 0; i < 32 / AT_ONCE; ++i) {
                    const int row = i * AT_ONCE + sub;
                    const long long o = __shfl_sync(~0u, off, row);
                    const int r = 32 * cw + row;
                    if (there)
                        tc_copy16(dst + r * 128 + (((piece & 7) ^ (r & 7)) << 4), src + (o >= 0 && inside ? 2 * o : -16 * piece),
                                  o >= 0 && inside);
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
                if (n >= LAG) {
                    tc_copies_wait<LAG>();
                    arrived(n - LAG);
                }
            }
        }
        tc_copies_wait<0>();
        if (ok)
            for (int n = max(0, 2 * tiles - LAG); n < 2 * tiles; ++n) arrived(n);
    } else if (warp == TC_WARPS - 1) {
        // ---- products ----
        if (lane == 0) {
            constexpr uint32_t SHAPE = 1u << 4 | (HALF ? 0u : 1u) << 7 | (HALF ? 0u : 1u) << 10 | (TC_ROWS >> 4) << 24;
            const uint32_t qk_shape = SHAPE | (TC_TILE >> 3) << 17;
            const uint32_t pv_shape = SHAPE | 1u << 16 | (uint32_t)(D16 >> 3) << 17;
            const uint64_t q_m = tc_matrix(tc_shared(q_s)), ring_m = tc_matrix(tc_shared(ring));
            const int steps = D16 / 16;
            bool ok = barrier_wait(&misc.q_full, 0, dead);
            tc_fence_after();
            auto scores = [&](int t) {  // S = Q K^T of tile t, smallest parts first
                const int n = 2 * t, slot = n % SLOTS;
                ok = ok && barrier_wait(&misc.full[slot], n / SLOTS & 1, dead);
                if (!ok) return;
                tc_fence_after();
                const uint64_t k_m = ring_m + slot * (S::SLOT >> 4);
                const uint32_t d = tmem + (t & 1) * 128;
                for (int p = QP - 1; p >= 0; --p)
                    for (int k = 0; k < steps; ++k) {
                        const uint64_t at = (k >> 2) * (TC_BLOCK >> 4) + (k & 3) * 2;
                        tc_product_shared(d, q_m + p * (NB * TC_BLOCK >> 4) + at, k_m + at, qk_shape, p < QP - 1 || k);
                    }
                tc_commit(&misc.empty[slot]);
                tc_commit(&misc.s_full[t & 1]);
            };
            scores(0);
            if (tiles > 1) scores(1);
            for (int t = 0; t < tiles && ok; ++t) {
                const int n = 2 * t + 1, slot = n % SLOTS, s = t & 1;
                ok = barrier_wait(&misc.full[slot], n / SLOTS & 1, dead) && barrier_wait(&misc.p_full[s], t >> 1 & 1, dead);
                if (!ok) break;
                tc_fence_after();
                const uint64_t v_m = ring_m + slot * (S::SLOT >> 4);
                const uint32_t o = tmem + 256 + s * 128, w = tmem + s * 128;
                // 16 positions a step: 8 columns of a weight part; 32 columns hold both
                // parts of 32 positions
                for (int k = 0; k < TC_TILE / 16; ++k)
                    for (int p = 1; p >= 0; --p)
                        tc_product_tensor(o, w + 32 * (k >> 1) + 16 * p + 8 * (k & 1), v_m + k * (2048 >> 4), pv_shape,
                                          t > 1 || k || p == 0);
                tc_commit(&misc.empty[slot]);
                if (t + 2 >= tiles) tc_commit(&misc.o_full[s]);  // the stream's last tile
                else scores(t + 2);
            }
            // nothing is in flight when the tensor memory is given back
            tc_commit(&misc.last);
            const uint64_t t0 = tc_nanoseconds();
            while (!barrier_try(&misc.last, 0) && tc_nanoseconds() - t0 < 100000000ull) {}
        }
        __syncwarp();
    } else {
        // ---- queries: fp32 -> 16-bit parts in shared memory, 16 rows by each warp ----
        {
            const int d = 4 * lane;
            const bool in_tile = d < NB * 64;
            const int es = a.x.dtype == BQ_F32 ? 4 : 2;
            const bool wide = a.x.q_row_stride % 4 == 0 && a.x.q_head_stride % 4 == 0 &&
                              (reinterpret_cast<uintptr_t>(a.x.q) & (4 * es - 1)) == 0;
#pragma unroll 4
            for (int k = 0; k < TC_ROWS / TC_SOFTMAX_WARPS; ++k) {
                const int i = warp + TC_SOFTMAX_WARPS * k, gr = first_row + i;
                float x[4] = {};
                if (gr < group_rows && d < D) {
                    const int row = (int)a.group.div((uint32_t)gr), head = h * G + gr - row * G;
                    const long long at = ((long long)first * R + row) * a.x.q_row_stride + head * a.x.q_head_stride + d;
                    if (a.x.dtype == BQ_F32) load_n<F32, 4>((const float *)a.x.q + at, wide, x);
                    else if (a.x.dtype == BQ_F16) load_n<F16, 4>((const __half *)a.x.q + at, wide, x);
                    else load_n<BF16, 4>((const __nv_bfloat16 *)a.x.q + at, wide, x);
                }
                float factor = a.scale_log2;
                if constexpr (HALF && QP > 1) {
                    // the largest of the row to [2^14, 2^15), as in the ordinary kernel
                    float top = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
                    int ex = (int)((__float_as_uint(top) >> 23) & 0xff) - 127;
                    if (top < 1.1754944e-38f || ex == 128) ex = 14;  // zero, subnormal or not finite: as it is
                    const int up = 14 - ex;
                    const float s1 = ldexpf(1.0f, up / 2), s2 = ldexpf(1.0f, up - up / 2);
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[e] = x[e] * s1 * s2;
                    factor = factor * ldexpf(1.0f, -(up / 2)) * ldexpf(1.0f, -(up - up / 2));
                }
                if (lane == 0) misc.factor[i] = factor;
                const int piece = (lane & 15) >> 1;
                uint8_t *to = q_s + (lane >> 4) * TC_BLOCK + i * 128 + ((piece ^ (i & 7)) << 4) + 8 * (lane & 1);
#pragma unroll
                for (int p = 0; p < QP; ++p) {
                    const uint2 w = make_uint2(tc_part<HALF>(x[0], x[1]), tc_part<HALF>(x[2], x[3]));
                    if (in_tile) *reinterpret_cast<uint2 *>(to + p * NB * TC_BLOCK) = w;
                }
            }
            fence_async_proxy();
            __syncwarp();
            if (lane == 0) barrier_arrive(&misc.q_full);
            asm volatile("bar.sync 1, 256;" ::: "memory");  // factors of all rows
        }

        // ---- weights of this stream's tiles ----
        const int s = warp >> 2, i = 32 * (warp & 3) + lane;  // this thread's row
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t s_at = tmem + lanes + s * 128, o_at = tmem + lanes + 256 + s * 128;
        const float factor = misc.factor[i];
        float ref = -INFINITY, l = 0.0f;
        bool ok = true;
        for (int t = s; t < tiles; t += 2) {
            ok = barrier_wait(&misc.mask_full[t % TC_MASKS], t / TC_MASKS & 1, dead) &&
                 barrier_wait(&misc.s_full[s], t >> 1 & 1, dead);
            if (!__all_sync(~0u, ok)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint4 m4 = *reinterpret_cast<const uint4 *>(misc.mask[t % TC_MASKS]);
            const uint32_t mask[4] = {m4.x, m4.y, m4.z, m4.w};
            uint32_t x[2][32];
            float top = -INFINITY;
            tc_load32(s_at, x[0]);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                tc_wait_load();
                if (c < 3) tc_load32(s_at + 32 * (c + 1), x[(c + 1) & 1]);
                const uint32_t(&y)[32] = x[c & 1];
                if (mask[c] == ~0u) {
                    float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int k = 0; k < 32; ++k) m[k & 3] = fmaxf(m[k & 3], __uint_as_float(y[k]) * factor);
                    top = fmaxf(top, fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])));
                } else {
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        if (mask[c] >> k & 1) top = fmaxf(top, __uint_as_float(y[k]) * factor);
                }
            }
            tc_load32(s_at, x[0]);
            const bool grows = top > ref + TC_GROWTH || (ref == -INFINITY && top > ref);
            const float now = grows ? top : ref;
            if (t > s && __any_sync(~0u, grows)) {
                const float alpha = grows ? tc_pow2(ref - now) : 1.0f;
                l *= alpha;
                tc_wait_load();
                for (int c = 0; c < D16; c += 32) {  // (columns from D16 on are not read)
                    tc_load32(o_at + c, x[1]);
                    tc_wait_load();
#pragma unroll
                    for (int k = 0; k < 32; ++k) x[1][k] = __float_as_uint(__uint_as_float(x[1][k]) * alpha);
                    tc_store32(o_at + c, x[1]);
                }
            }
            ref = now;
            const float shift = (HALF ? (float)TC_SHIFT_F16 : 0.0f) - (ref == -INFINITY ? 0.0f : ref);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                tc_wait_load();
                if (c < 3) tc_load32(s_at + 32 * (c + 1), x[(c + 1) & 1]);
                uint32_t(&y)[32] = x[c & 1];
                uint32_t w[32];
                float sum[2] = {0.0f, 0.0f};
#pragma unroll
                for (int k = 0; k < 32; k += 2) {
                    float u = tc_pow2(fmaf(__uint_as_float(y[k]), factor, shift));
                    float v = tc_pow2(fmaf(__uint_as_float(y[k + 1]), factor, shift));
                    if (mask[c] != ~0u) {
                        if (!(mask[c] >> k & 1)) u = 0.0f;
                        if (!(mask[c] >> (k + 1) & 1)) v = 0.0f;
                    }
                    sum[0] += u, sum[1] += v;
                    w[k / 2] = tc_part<HALF>(u, v);
                    w[16 + k / 2] = tc_part<HALF>(u, v);
                }
                l += sum[0] + sum[1];
                tc_store32(s_at + 32 * c, w);
            }
            tc_wait_store();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) barrier_arrive(&misc.p_full[s]);
        }

        // ---- join of the streams, in the ring's place: nothing reads or fills it once
        // the last products of both are complete ----
        const int last = tiles > 1 ? 2 : 1;
        for (int k = 0; k < last; ++k) ok = ok && barrier_wait(&misc.o_full[k], 0, dead);
        ok = __all_sync(~0u, ok);
        tc_fence_after();
        // partial results of the ordinary kernel carry 2^ATTN_SHIFT_F16 over fp16 caches
        constexpr float LIKE = HALF ? (float)(1 << (ATTN_SHIFT_F16 - TC_SHIFT_F16)) : 1.0f;
        float *row = reinterpret_cast<float *>(ring) + i * S::OROW;
        if (s == 1 && last == 2) {
            for (int c = 0; c < D16 && ok; c += 32) {
                uint32_t x[32];
                tc_load32(o_at + c, x);
                tc_wait_load();
#pragma unroll
                for (int k = 0; k < 32; k += 4)
                    *reinterpret_cast<float4 *>(row + c + k) =
                        make_float4(__uint_as_float(x[k]), __uint_as_float(x[k + 1]), __uint_as_float(x[k + 2]),
                                    __uint_as_float(x[k + 3]));
            }
            misc.ml[i] = make_float2(ref, l);
        }
        asm volatile("bar.sync 1, 256;" ::: "memory");
        const long long unit = (((long long)g * a.max_chunks + ck) * KVH + h) * a.row_tiles + rt;
        if (s == 0) {
            const float2 o = last == 2 ? misc.ml[i] : make_float2(-INFINITY, 0.0f);
            const float top = fmaxf(ref, o.x);
            const float f = ref == -INFINITY ? 0.0f : LIKE * tc_pow2(ref - top);
            const float e = o.x == -INFINITY ? 0.0f : LIKE * tc_pow2(o.x - top);
            for (int c = 0; c < D16 && ok; c += 32) {
                uint32_t x[32];
                tc_load32(o_at + c, x);
                tc_wait_load();
#pragma unroll
                for (int k = 0; k < 32; k += 4) {
                    float4 v = last == 2 ? *reinterpret_cast<const float4 *>(row + c + k) : make_float4(0, 0, 0, 0);
                    v.x = fmaf(f, __uint_as_float(x[k]), e * v.x);
                    v.y = fmaf(f, __uint_as_float(x[k + 1]), e * v.y);
                    v.z = fmaf(f, __uint_as_float(x[k + 2]), e * v.z);
                    v.w = fmaf(f, __uint_as_float(x[k + 3]), e * v.w);
                    *reinterpret_cast<float4 *>(row + c + k) = v;
                }
            }
            if (first_row + i < group_rows) a.part_ml[unit * TC_ROWS + i] = make_float2(top, fmaf(f, l, e * o.y));
        }
        asm volatile("bar.sync 1, 256;" ::: "memory");
        if (4 * lane < D) {
            float *dst = a.part_o + unit * TC_ROWS * D + 4 * lane;
            const float *src = reinterpret_cast<const float *>(ring) + 4 * lane;
            for (int r = warp; r < TC_ROWS && first_row + r < group_rows; r += TC_SOFTMAX_WARPS)
                *reinterpret_cast<float4 *>(dst + r * D) = *reinterpret_cast<const float4 *>(src + r * S::OROW);
        }
        tc_fence_before();
    }
    __syncthreads();
    if (warp == TC_WARPS - 1) {
        tc_fence_after();
        if (*dead && lane == 0) atomicOr(status, BQ_DEVERR_WAIT);
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(TC_COLUMNS) : "memory");
    }
}

template <bool HALF, int QP, int NB>
cudaError_t prefix_launch_of(const AttnArgs &a, int grid, void *stream, unsigned int *status) {
    auto *kern = prefix_kernel<HALF, QP, NB>;
    constexpr int smem = TcShape<QP, NB>::SMEM;
    static std::atomic<bool> ready[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!ready[dev].load()) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        ready[dev].store(true);
    }
    return launch_pdl(kern, dim3((unsigned)grid), TC_WARPS * 32, smem, stream, 1, a, status);
}
template <bool HALF, int QP>
cudaError_t prefix_launch(const AttnArgs &a, int grid, void *stream, unsigned int *status) {
    return a.c.head_dim <= 64 ? prefix_launch_of<HALF, QP, 1>(a, grid, stream, status)
                              : prefix_launch_of<HALF, QP, 2>(a, grid, stream, status);
}

}  // namespace bq
