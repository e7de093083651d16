// bq_attn.cuh -- attention of a request's last one to six tokens over its paged
// key-value cache (bq_paged_attention in include/bqgemv.h).
//
// Mathematics.  Per query row: s_t = scale q.k_t, o = sum_t e^(s_t) v_t / sum_t e^(s_t)
// in one pass over the cache with a running maximum m and sum l: a tile with
// maximum m' rescales what was summed by 2^(m - m') (all exponents in base 2,
// the factor log2 e folded into scale).  The positions are cut into chunks of
// a fixed length, each chunk's tiles are shared by four warps, and the partial
// (m, l, O) are joined in a fixed order: the warps' in shared memory, the
// chunks' over a thread-block cluster where the table holds few of them (the
// call is one launch), else in a second kernel.  Which chunks exist depends on the geometry and
// the length alone, and an empty chunk joins with weight zero, so a row's bits
// depend on its own inputs and the geometry only.  The largest score's weight is 1
// (2^SHIFT), so l is 0 for a row that sees nothing and for no other: it gives 0.
//
// Bound by HBM: every live byte of the cache is read once (again per 8 NT query
// rows of a kv head, through L2), about 4 flop per byte and query row.  Measured:
// 48 requests to 12001 positions, bf16, 32 heads over 8, 1.32 GB: 202 us, 6.5 TB/s;
// one request of 100003, fp16: 41 us, 5.0 TB/s; Q8_0 is bound by instructions
// (48 requests to 6000, bf16 queries: 92 us, 3.9 TB/s; 5 rows of 40 heads over 8 at
// 24577: 53 us).
// So the kernel is built around the loads:
//  - Every warp has a ring of STAGES tiles of K and V rows in shared memory
//    that it fills itself by 16-byte asynchronous copies (any page size and
//    stride; what is not there is filled with zeros), STAGES - 1 tiles ahead of
//    the one it works on: about 16 KB in flight per warp, 128 KB per SM, with no
//    barrier between warps.  Rows are swizzled by 16-byte pieces, so that every read of
//    a matrix operand is free of bank conflicts.
//  - S^T = K Q^T has positions as rows and is summed over d; O^T = V^T P^T has d
//    as rows and is summed over positions, V read with ldmatrix's transpose.
//    So K and V are the 16-row operand and the query rows of a kv head (all
//    heads of its group, all new tokens) the 8-column one: 8 rows per n-tile.
//    The scores come out with positions along the lanes' r, the weights go in
//    with positions along c: movmatrix transposes the 8 x 8 tile in registers.
//  - tcgen05 would hold 128 rows of accumulator for 1 to 48 query rows; with 8
//    query rows per n-tile mma.sync's pipe is about a fifth busy at HBM speed.
// Precision.  The tensor cores multiply 16-bit values exactly.  A query of
// the cache's own type is used as it is; any other is split into QP 16-bit
// parts (fp16: 2 parts, 22 bits, after scaling the row by a power of two, which
// lets a bf16 query through in one; bf16: 3 parts, 24 bits), the weights into PP
// parts: 2 of fp16 (off by 2^-23 of them), 3 of bf16 (24 bits).  Fewer parts show in a
// 16-bit output: with two of bf16 (17 bits) 0.2% of its values were not the nearest
// ones, with three 0.02% are not, plain fp32 sums leave 0.09% (48 requests to 12001:
// 202 us against 201; 40 to 5000, 32 heads of 64 over one: 28 against 24, the 32-row
// tile spills); with one of fp16, bf16 queries over Q8_0, 8.9% were not (8 requests to
// 4000; 48 to 6000: 92 us against 85).  Each tile's products
// are summed by the tensor core from zero, smallest parts first, and added to
// the fp32 accumulator by an fp32 FMA, since the tensor core truncates its sums.
// Q8_0 codes are exact in fp16; a key's scale multiplies its block's partial
// score, a value's scale its weight, both in fp32 before any rounding to parts.
#pragma once

#include <atomic>
#include <cmath>
#include <type_traits>

#include "bq_attn.h"

namespace bq {

enum { KV_F16 = 0, KV_BF16 = 1, KV_Q8 = 2 };

template <int N>
struct Words {
    uint32_t w[N];
};

// asynchronous copy of 16 (4, 8) bytes to shared memory, zeros where !ok
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const void *src, bool ok) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(ok ? 8 : 0) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t smem_address(const void *p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ uint4 ldmatrix4(uint32_t at) {
    uint4 v;
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(at)
                 : "memory");
    return v;
}
__device__ __forceinline__ uint4 ldmatrix4_trans(uint32_t at) {
    uint4 v;
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(at)
                 : "memory");
    return v;
}

// d = a b + d on the tensor cores; FROM_ZERO: d = a b
template <bool HALF, bool FROM_ZERO = false>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint4 &a, uint32_t b0, uint32_t b1) {
    const float c0 = FROM_ZERO ? 0.0f : d[0], c1 = FROM_ZERO ? 0.0f : d[1], c2 = FROM_ZERO ? 0.0f : d[2],
                c3 = FROM_ZERO ? 0.0f : d[3];
    if constexpr (HALF)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%10,%11,%12,%13};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%10,%11,%12,%13};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

// 2^x by the hardware's approximation (2 ulp; below 2^-126: 0)
__device__ __forceinline__ float pow2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t o;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(o) : "r"(v));
    return o;
}

// two fp32 values as PARTS packed pairs of 16-bit values that add up to them,
// each part the rest's value rounded to nearest
template <bool HALF, int PARTS>
__device__ __forceinline__ Words<PARTS> split_pair(float x, float y) {
    Words<PARTS> o;
#pragma unroll
    for (int p = 0; p < PARTS; ++p) {
        if constexpr (HALF) {
            const __half2 h = __floats2half2_rn(x, y);
            o.w[p] = *reinterpret_cast<const uint32_t *>(&h);
            if (p + 1 < PARTS) {
                const float2 f = __half22float2(h);
                x -= f.x;
                y -= f.y;
            }
        } else {
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o.w[p]) : "f"(y), "f"(x));
            if (p + 1 < PARTS) {
                x -= __uint_as_float(o.w[p] << 16);
                y -= __uint_as_float(o.w[p] & 0xffff0000u);
            }
        }
    }
    return o;
}

// Four int8 codes as two pairs of fp16.  With b = code + 128 (the sign bit
// turned) 0x6400 | b is 1024 + b, a whole number that fp16 holds; less 1152 it
// is the code, exact.
__device__ __forceinline__ uint2 codes_to_f16(uint32_t w) {
    uint2 o;
    w ^= 0x80808080u;
    const uint32_t lo = __byte_perm(w, 0x64646464u, 0x4140), hi = __byte_perm(w, 0x64646464u, 0x4342);
    asm("sub.f16x2 %0, %1, %2;" : "=r"(o.x) : "r"(lo), "r"(0x64806480u));
    asm("sub.f16x2 %0, %1, %2;" : "=r"(o.y) : "r"(hi), "r"(0x64806480u));
    return o;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// a word of shared memory of another CTA of the cluster
__device__ __forceinline__ float peer_float(uint32_t at, int rank) {
    float v;
    asm volatile(
        "{\n\t.reg .b32 p;\n\tmapa.shared::cluster.u32 p, %1, %2;\n\tld.shared::cluster.f32 %0, [p];\n\t}"
        : "=f"(v)
        : "r"(at), "r"(rank)
        : "memory");
    return v;
}

// element d of query row g (of the rows of kv head h) of request b
__device__ __forceinline__ void attn_store(const AttnArgs &a, int b, int h, int g, int d, float v) {
    const int row = (int)a.group.div((uint32_t)g);
    const int head = h * (int)a.group.d + g - row * (int)a.group.d;
    const long long at = ((long long)b * a.x.rows + row) * a.x.out_row_stride + head * a.x.out_head_stride + d;
    if (a.x.dtype == BQ_F32) ((float *)a.x.out)[at] = v;
    else if (a.x.dtype == BQ_F16) ((__half *)a.x.out)[at] = __float2half_rn(v);
    else ((__nv_bfloat16 *)a.x.out)[at] = __float2bfloat16_rn(v);
}

template <int KV, int QP, int PP, int DP, int NT>
struct AttnShape {
    static constexpr bool Q8 = KV == KV_Q8, HALF = KV != KV_BF16;
    static constexpr int ROWS = 8 * NT;
    static constexpr int WARPS = ATTN_WARPS;
    // 16 positions per tile (32 of short rows) whatever NT: the order of the sums, and so a row's
    // bits, must not depend on how many rows are computed beside it
    static constexpr int TT = DP <= 64 || (Q8 && DP <= 128) ? 2 : 1, TILE = 16 * TT;
    static constexpr int ROWB = Q8 ? DP : 2 * DP;  // bytes of a row in the ring
    static constexpr int SCALEB = Q8 ? (DP / 32 + 1) / 2 * 4 : 0;  // words of a row's scales
    static constexpr int STAGE = 2 * TILE * (ROWB + SCALEB) + 4 * TILE;
    static constexpr int OROW = DP + 4;  // floats: 8 lanes r and 4 row pairs c in 32 banks
    // query rows: 16 bytes apart modulo 128 for ldmatrix; 64 for the Q8_0 order,
    // where 8 lanes read 16-byte pieces of 2 rows
    static constexpr int QROW = 2 * DP + (Q8 ? 64 : 16);
    static constexpr int Q_BYTES = QP * ROWS * QROW;
    // a warp's ring holds its O for the join once its tiles are done
    static constexpr int ring_of(int stages) {
        return stages * STAGE > ROWS * OROW * 4 ? stages * STAGE : ROWS * OROW * 4;
    }
    static constexpr int smem_of(int stages) {
        return WARPS * ring_of(stages) + Q_BYTES + (2 * WARPS + 1) * ROWS * 4;
    }
    static constexpr int most_stages(int limit) {
        int n = 6;
        while (n > 1 && smem_of(n) > limit) --n;
        return n;
    }
    // Two CTAs per SM where two stages fit (the scan of 1024 requests besides),
    // else one, with the scan of the most requests.  Three with heads of up to 64
    // and one n-tile (160 requests to 2500 positions: 34 us against 43; with heads
    // of 128 and two stages left, 217 against 209 for 48 requests to 12001).
    static constexpr int OCC = DP <= 64 && NT == 1 && most_stages(74 * 1024) >= 2 ? 3
                               : most_stages(108 * 1024) >= 2                     ? 2
                                                                                  : 1;
    static constexpr int STAGES = most_stages(OCC == 3 ? 74 * 1024 : OCC == 2 ? 108 * 1024 : 209 * 1024);
    static constexpr int RING = ring_of(STAGES), SMEM = smem_of(STAGES);
    static_assert(STAGES >= 2 && RING % 16 == 0 && STAGE % 16 == 0 && TILE > BQ_VERIFY_MAX_ROWS);
};

template <int KV, int QP, int PP, int DP, int NT, bool MODES>
__global__ void __launch_bounds__(AttnShape<KV, QP, PP, DP, NT>::WARPS * 32, AttnShape<KV, QP, PP, DP, NT>::OCC)
    attn_kernel(const __grid_constant__ AttnArgs a, unsigned int *status) {
    using S = AttnShape<KV, QP, PP, DP, NT>;
    constexpr bool Q8 = S::Q8, HALF = S::HALF;
    constexpr int TT = S::TT, ROWS = S::ROWS, TILE = S::TILE, STAGES = S::STAGES, ROWB = S::ROWB;
    constexpr int WARPS = S::WARPS;
    const int mode = MODES ? a.mode : (int)ATTN_ALL;  // (known, it costs the ordinary calls nothing)
    constexpr int MT = DP / 16;  // 16-row tiles of O^T
    constexpr float SHIFT = HALF ? (float)ATTN_SHIFT_F16 : 0.0f;
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t *q_s = smem + WARPS * S::RING;
    float *m_s = reinterpret_cast<float *>(q_s + S::Q_BYTES), *l_s = m_s + WARPS * ROWS;
    float *f_s = l_s + WARPS * ROWS;            // per row: factor of its scores
    int *pre = reinterpret_cast<int *>(f_s + ROWS);  // [requests + 1]
    __shared__ int scan_s[WARPS];

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = lane >> 2, c = lane & 3;
    uint8_t *ring = smem + warp * S::RING;
    const int B = a.x.requests, R = a.x.rows, D = a.c.head_dim, KVH = a.c.kv_heads;
    const int most = a.x.table_width * a.c.page_size;
    pdl_wait();
    const bool parts = mode == ATTN_REST || mode == ATTN_PREFIX;  // partial results alone
    if ((a.max_chunks > 1 && !a.cluster) || parts) pdl_launch_dependents();

    const bool shared = mode == ATTN_PREFIX;
    // pages that request b shares
    auto common = [&](int b) {
        int g = 0;
        while (a.group_end[g] <= b) ++g;  // ends: the groups cover the requests
        return a.group_pages[g];
    };
    // pages before the first position that this launch covers of request b
    auto skipped = [&](int b) { return mode == ATTN_REST ? common(b) : 0; };
    auto length = [&](int b) {
        if (shared) return a.group_pages[b] * a.c.page_size;
        const int n = attn_clamped(a.x.lens[b], most);
        if (mode == ATTN_ALL) return n;
        const int before = common(b) * a.c.page_size, rest = attn_rest(n, R, before);
        return mode == ATTN_REST ? rest : attn_sees(n, R, before) ? n : 0;
    };
    const long long per_chunk = (long long)KVH * a.row_tiles;
    // direct: a CTA per unit that the table can hold, units beyond a request's
    // length are empty.  Else a CTA takes every gridDim.x-th live unit, which
    // exclusive prefix sums of the requests' units tell.
    const bool direct = a.direct;
    auto checked = [&](int b) {
        if (shared) return;
        const int len = a.x.lens[b];
        if (len < 0 || len > most || (len && mode != ATTN_ALL && !attn_sees(len, R, common(b) * a.c.page_size)))
            atomicOr(status, BQ_DEVERR_LENGTH);
    };
    if (!direct) {
        const int per = (B + WARPS * 32 - 1) / (WARPS * 32);
        const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
        int n = 0;
        for (int b = b0; b < b1; ++b) {
            if (blockIdx.x == 0) checked(b);
            n += attn_chunks(length(b), a.chunk);
        }
        int v = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(~0u, v, o);
            if (lane >= o) v += u;
        }
        if (lane == 31) scan_s[warp] = v;
        __syncthreads();
        int excl = v - n;
        for (int w = 0; w < warp; ++w) excl += scan_s[w];
        for (int b = b0; b < b1; ++b) {
            pre[b] = excl;
            excl += attn_chunks(length(b), a.chunk);
        }
        if (b0 < B && b1 == B) pre[B] = excl;
        __syncthreads();
    }
    const long long units = direct ? gridDim.x : pre[B] * per_chunk;

    for (long long u = blockIdx.x; u < units; u += gridDim.x) {
        int b = 0, hr, ck;
        if (direct) {
            // a cluster's units are neighbours; else all requests' first chunks come
            // first, the ragged last ones fill the gaps
            const uint32_t pairs = (uint32_t)B * (uint32_t)per_chunk;
            const uint32_t q = (uint32_t)u / (a.cluster ? (uint32_t)a.max_chunks : pairs);
            const uint32_t m = (uint32_t)u - q * (a.cluster ? (uint32_t)a.max_chunks : pairs);
            const uint32_t rest = a.cluster ? q : m;
            ck = (int)(a.cluster ? m : q);
            b = (int)(rest / (uint32_t)per_chunk);
            hr = (int)(rest - (uint32_t)b * (uint32_t)per_chunk);
        } else {
            const int cu = (int)(u / per_chunk);
            hr = (int)(u - cu * per_chunk);
            for (int hi = B; hi - b > 1;) {
                const int mid = (b + hi) >> 1;
                if (pre[mid] <= cu) b = mid;
                else hi = mid;
            }
            ck = cu - pre[b];
        }
        const int h = hr / a.row_tiles, rt = hr - h * a.row_tiles;
        const int begin = ck * a.chunk, first_row = rt * ROWS;
        // ATTN_PREFIX: the group's requests, and the first of them that holds the
        // shared pages, whose table row tells them
        int first = b, owner = b, group_rows = a.group_rows;
        if (shared) {
            first = b ? a.group_end[b - 1] : 0;
            group_rows = (a.group_end[b] - first) * R * (int)a.group.d;
            owner = 0x7fffffff;
            for (int i = first + lane; i < a.group_end[b] && owner == 0x7fffffff; i += 32)
                if (attn_sees(attn_clamped(a.x.lens[i], most), R, length(b))) owner = i;
            owner = __reduce_min_sync(~0u, owner);
            if (first_row >= group_rows || owner == 0x7fffffff) continue;  // nobody reads its partial results
        }

        // ---- loads whose addresses do not wait for the length: table entries
        // (there is one for every position of the table), queries ----
        const int *row_table = a.x.table + owner * a.x.table_stride + skipped(b);
        const int mine = lane & (TILE - 1);  // the position of a tile that this lane looks up
        const int chunk_end = min(begin + a.chunk, most - skipped(b) * a.c.page_size);
        auto entry_of = [&](int t) { return t < chunk_end ? row_table[a.page.div((uint32_t)t)] : -1; };
        int entry = entry_of(begin + warp * TILE + mine);
        float qx[ROWS / WARPS][DP / 32];
#pragma unroll
        for (int k = 0; k < ROWS / WARPS; ++k) {
            const int g = first_row + warp + WARPS * k;
            const int row = (int)a.group.div((uint32_t)g);
            const int head = h * (int)a.group.d + g - row * (int)a.group.d;
            const long long at = ((long long)first * R + row) * a.x.q_row_stride + head * a.x.q_head_stride;
#pragma unroll
            for (int e = 0; e < DP / 32; ++e) {
                const int d = lane + 32 * e;
                qx[k][e] = d >= D || g >= group_rows ? 0.0f
                           : a.x.dtype == BQ_F32       ? ((const float *)a.x.q)[at + d]
                           : a.x.dtype == BQ_F16       ? __half2float(((const __half *)a.x.q)[at + d])
                                                       : __bfloat162float(((const __nv_bfloat16 *)a.x.q)[at + d]);
            }
        }
        const int len = length(b), end = min(len, begin + a.chunk);
        if (direct) {
            if (ck == 0 && hr == 0 && tid == 0) checked(b);
            if (!a.cluster && ck >= attn_chunks(len, a.chunk)) continue;
        }

        // ---- the ring: tile `t0` of this warp into stage `st` ----
        const long long head_off = (long long)h * a.c.head_stride;
        auto fill = [&](int t0, int entry, int st) {
            const int t = t0 + mine;
            long long off = -1;  // element offset, -1 where there is nothing to read
            if (t < end) {
                if (entry >= 0 && entry < a.c.pages) {
                    const uint32_t in_page = (uint32_t)t - a.page.div((uint32_t)t) * a.page.d;
                    off = entry * a.c.page_stride + in_page * a.c.slot_stride + head_off;
                } else {
                    atomicOr(status, BQ_DEVERR_PAGE);
                }
            }
            const uint32_t base = smem_address(ring) + st * S::STAGE;
            int *meta = reinterpret_cast<int *>(ring + st * S::STAGE + 2 * TILE * (ROWB + S::SCALEB));
            // -1: nothing there; else the first scale's place in its word
            if (lane < TILE) meta[lane] = off < 0 ? -1 : (int)((off >> 5) & 1);
            constexpr int PIECES = ROWB / 16;       // of a row
            constexpr int ROWS_AT_ONCE = 32 / PIECES > 0 ? 32 / PIECES : 1;
            static_assert(PIECES <= 32);
            const int piece = lane % PIECES;
            const bool inside = piece * (Q8 ? 16 : 8) < D;
#pragma unroll
            for (int i = 0; i < TILE / ROWS_AT_ONCE; ++i) {
                const int row = i * ROWS_AT_ONCE + lane / PIECES;
                const long long o = __shfl_sync(~0u, off, row);
                const bool ok = o >= 0 && inside;
                const long long at = ok ? (Q8 ? o : 2 * o) + 16 * piece : 0;
                const int kk = Q8 ? ((row & 3) << 1 | (row >> 2 & 1)) : row & 7;
                copy16(base + row * ROWB + ((piece ^ (kk & (PIECES - 1))) << 4), (const uint8_t *)a.c.k + at, ok);
                copy16(base + (TILE + row) * ROWB + ((piece ^ (row & 7 & (PIECES - 1))) << 4),
                       (const uint8_t *)a.c.v + at, ok);
            }
            if constexpr (Q8) {
                const int nb = D >> 5;  // scales of a row; an odd number of them may start mid-word
                const uint32_t sk = base + 2 * TILE * ROWB + mine * S::SCALEB, sv = sk + TILE * S::SCALEB;
                const long long so = off < 0 ? 0 : off >> 5;
                const uint8_t *ks = (const uint8_t *)a.c.k_scale + (so & ~1ll) * 2;
                const uint8_t *vs = (const uint8_t *)a.c.v_scale + (so & ~1ll) * 2;
                if (lane < TILE) {
                    if (nb % 4 == 0) {
#pragma unroll
                        for (int i = 0; i < (DP + 127) / 128; ++i)
                            if (4 * i < nb) {
                                copy8(sk + 8 * i, ks + 8 * i, off >= 0);
                                copy8(sv + 8 * i, vs + 8 * i, off >= 0);
                            }
                    } else {
                        const int bytes = 2 * nb + 2 * (int)(so & 1);
#pragma unroll
                        for (int i = 0; i < S::SCALEB / 4; ++i) {
                            const int n = off < 0 ? 0 : min(4, max(0, bytes - 4 * i));
                            copy4(sk + 4 * i, n ? ks + 4 * i : ks, n);
                            copy4(sv + 4 * i, n ? vs + 4 * i : vs, n);
                        }
                    }
                }
            }
        };

        const int stride = WARPS * TILE;
        int tile = begin + warp * TILE;
        int ahead = tile;  // the next tile to fetch
#pragma unroll
        for (int st = 0; st < STAGES - 1; ++st) {
            if (ahead < end) {
                const int now = entry;
                entry = entry_of(ahead + stride + mine);
                fill(ahead, now, st);
            }
            copies_commit();
            ahead += stride;
        }

        // ---- queries: fp32 -> 16-bit parts in shared memory ----
#pragma unroll
        for (int k = 0; k < ROWS / WARPS; ++k) {
            const int i = warp + WARPS * k;
            float(&x)[DP / 32] = qx[k];
            float top = 0.0f;
#pragma unroll
            for (int e = 0; e < DP / 32; ++e) top = fmaxf(top, fabsf(x[e]));
            float factor = a.scale_log2;
            if constexpr (HALF && (QP > 1 || Q8)) {
                // the largest of the row to [2^14, 2^15): the second part of anything
                // down to 2^-29 of it is still a normal fp16 number
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
                int ex = (int)((__float_as_uint(top) >> 23) & 0xff) - 127;
                if (top < 1.1754944e-38f || ex == 128) ex = 14;  // zero, subnormal or not finite: as it is
                const int up = 14 - ex;
                const float s1 = ldexpf(1.0f, up / 2), s2 = ldexpf(1.0f, up - up / 2);
#pragma unroll
                for (int e = 0; e < DP / 32; ++e) x[e] = x[e] * s1 * s2;
                factor = factor * ldexpf(1.0f, -(up / 2)) * ldexpf(1.0f, -(up - up / 2));
            }
            if (lane == 0) f_s[i] = factor;
#pragma unroll
            for (int e = 0; e < DP / 32; ++e) {
                const Words<QP> w = split_pair<HALF, QP>(x[e], 0.0f);
#pragma unroll
                for (int p = 0; p < QP; ++p)
                    *reinterpret_cast<uint16_t *>(q_s + (p * ROWS + i) * S::QROW + 2 * (lane + 32 * e)) =
                        (uint16_t)w.w[p];
            }
        }
        __syncthreads();

        // positions that this thread's query rows see, and their factors
        int lim[NT][2];
        float fac[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int i = 8 * nt + 2 * c + x, g = first_row + i;
                lim[nt][x] = g >= group_rows ? 0 : shared ? len : len - R + (int)a.group.div((uint32_t)g) + 1;
                fac[nt][x] = f_s[i];
            }

        float O[MT][NT][4], m[NT][2], l[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt][0] = m[nt][1] = -INFINITY;
            l[nt][0] = l[nt][1] = 0.0f;
#pragma unroll
            for (int v = 0; v < MT; ++v)
#pragma unroll
                for (int x = 0; x < 4; ++x) O[v][nt][x] = 0.0f;
        }

        // Q8_0: a weight times its value's scale goes into fp16.  It is divided by
        // 2^vexp, which bounds the scales seen so far from above, and so is O; a
        // larger scale than before rescales O along with alpha.  -14: fp16's least
        // normal exponent.  vend: the same per query row after the last tile.
        [[maybe_unused]] int vexp = -14, vend[NT][2];
        [[maybe_unused]] bool ended = false;
        for (int st = 0; tile < end; tile += stride, st = st + 1 == STAGES ? 0 : st + 1) {
            copies_wait<STAGES - 2>();  // this tile's copies have landed,
            __syncwarp();               // every lane's, and every lane is done with the tile before
            {
                const int into = st == 0 ? STAGES - 1 : st - 1;
                if (ahead < end) {
                    const int now = entry;
                    entry = entry_of(ahead + stride + mine);
                    fill(ahead, now, into);
                }
                copies_commit();
                ahead += stride;
            }
            const uint8_t *k_s = ring + st * S::STAGE, *v_s = k_s + TILE * ROWB;
            const uint8_t *ks_s = v_s + TILE * ROWB, *vs_s = ks_s + TILE * S::SCALEB;
            const int *meta = reinterpret_cast<const int *>(vs_s + TILE * S::SCALEB);
            int there[TT][2];
#pragma unroll
            for (int s = 0; s < TT; ++s)
#pragma unroll
                for (int y = 0; y < 2; ++y) there[s][y] = meta[16 * s + 8 * y + r];
            // Q8_0: the scales of this thread's positions, a word holds two; a row of an
            // odd number of scales may start in the middle of a word
            constexpr int SW = S::SCALEB / 4 > 0 ? S::SCALEB / 4 : 1;
            [[maybe_unused]] auto scales_of = [&](const uint8_t *base, int s, int y, uint32_t(&w)[SW]) {
                const uint8_t *at = base + (16 * s + 8 * y + r) * S::SCALEB;
                if constexpr (SW % 2 == 0) {
#pragma unroll
                    for (int i = 0; i < SW / 2; ++i) {
                        const uint2 v = *reinterpret_cast<const uint2 *>(at + 8 * i);
                        w[2 * i] = v.x, w[2 * i + 1] = v.y;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < SW; ++i) w[i] = *reinterpret_cast<const uint32_t *>(at + 4 * i);
                }
                if ((D >> 5) & 1) {
                    const int shift = 16 * max(there[s][y], 0);
#pragma unroll
                    for (int i = 0; i < SW; ++i) w[i] = __funnelshift_r(w[i], i + 1 < SW ? w[i + 1] : 0u, shift);
                    // (a word's last half is no scale of this row, and its values are 0)
                }
            };
            [[maybe_unused]] auto scale = [](const uint32_t(&w)[SW], int j) {
                return __half2float(__ushort_as_half((unsigned short)(w[j >> 1] >> (16 * (j & 1)))));
            };

            // ---- scores ----
            float sc[TT][NT][4];
            if constexpr (Q8) {
#pragma unroll
                for (int s = 0; s < TT; ++s)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int x = 0; x < 4; ++x) sc[s][nt][x] = 0.0f;
                uint32_t kw[TT][2][SW];
#pragma unroll
                for (int s = 0; s < TT; ++s)
#pragma unroll
                    for (int y = 0; y < 2; ++y) scales_of(ks_s, s, y, kw[s][y]);
#pragma unroll
                for (int j = 0; j < DP / 32; ++j) {
                    uint4 lo[TT], hi[TT];  // the operand over the pieces' first and second 4 codes
                    float d[TT][2];
#pragma unroll
                    for (int s = 0; s < TT; ++s) {
                        uint2 f[2], g[2];
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const int row = 16 * s + 8 * y + r;
                            const int key = ((r & 3) << 1 | (r >> 2 & 1)) & (ROWB / 16 - 1);
                            const uint2 w = *reinterpret_cast<const uint2 *>(
                                k_s + row * ROWB + (((2 * j + (c >> 1)) ^ key) << 4) + 8 * (c & 1));
                            f[y] = codes_to_f16(w.x);
                            g[y] = codes_to_f16(w.y);
                            d[s][y] = scale(kw[s][y], j);
                        }
                        lo[s] = make_uint4(f[0].x, f[1].x, f[0].y, f[1].y);
                        hi[s] = make_uint4(g[0].x, g[1].x, g[0].y, g[1].y);
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float t[TT][4];  // smallest parts first
#pragma unroll
                        for (int p = QP - 1; p >= 0; --p) {
                            const uint4 q = *reinterpret_cast<const uint4 *>(
                                q_s + (p * ROWS + 8 * nt + r) * S::QROW + 16 * (c + 4 * j));
#pragma unroll
                            for (int s = 0; s < TT; ++s) {
                                if (p == QP - 1) mma16816<HALF, true>(t[s], lo[s], q.x, q.y);
                                else mma16816<HALF>(t[s], lo[s], q.x, q.y);
                                mma16816<HALF>(t[s], hi[s], q.z, q.w);
                            }
                        }
#pragma unroll
                        for (int s = 0; s < TT; ++s)
#pragma unroll
                            for (int x = 0; x < 4; ++x) sc[s][nt][x] = fmaf(d[s][x >> 1], t[s][x], sc[s][nt][x]);
                    }
                }
            } else {
                // a sum per part and parity of the step: short chains, added smallest first
                float t[2][QP][TT][NT][4];
                const int krow = (lane & 7) + (lane >> 3 & 1) * 8;
                const uint32_t k_at = smem_address(k_s) + krow * ROWB;
                const uint32_t q_at = smem_address(q_s) + (lane & 7) * S::QROW + (lane >> 3) * 16;
#pragma unroll
                for (int j = 0; j < DP / 32; ++j) {
                    uint4 k0[TT], k1[TT];
#pragma unroll
                    for (int s = 0; s < TT; ++s) {
                        k0[s] = ldmatrix4(k_at + 16 * s * ROWB + (((4 * j + (lane >> 4)) ^ (krow & 7)) << 4));
                        k1[s] = ldmatrix4(k_at + 16 * s * ROWB + (((4 * j + 2 + (lane >> 4)) ^ (krow & 7)) << 4));
                    }
#pragma unroll
                    for (int p = 0; p < QP; ++p)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const uint4 q = ldmatrix4(q_at + (p * ROWS + 8 * nt) * S::QROW + 64 * j);
#pragma unroll
                            for (int s = 0; s < TT; ++s) {
                                if (j == 0) {
                                    mma16816<HALF, true>(t[0][p][s][nt], k0[s], q.x, q.y);
                                    mma16816<HALF, true>(t[1][p][s][nt], k1[s], q.z, q.w);
                                } else {
                                    mma16816<HALF>(t[0][p][s][nt], k0[s], q.x, q.y);
                                    mma16816<HALF>(t[1][p][s][nt], k1[s], q.z, q.w);
                                }
                            }
                        }
                }
#pragma unroll
                for (int s = 0; s < TT; ++s)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            float sum = t[0][QP - 1][s][nt][x] + t[1][QP - 1][s][nt][x];
#pragma unroll
                            for (int p = QP - 2; p >= 0; --p) sum += t[0][p][s][nt][x] + t[1][p][s][nt][x];
                            sc[s][nt][x] = sum;
                        }
            }

            // ---- softmax weights ----
            float alpha[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float top = -INFINITY;
#pragma unroll
                    for (int s = 0; s < TT; ++s)
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const int t = tile + 16 * s + 8 * y + r;
                            float &v = sc[s][nt][2 * y + x];
                            v = t < lim[nt][x] && there[s][y] >= 0 ? v * fac[nt][x] : -INFINITY;
                            top = fmaxf(top, v);
                        }
                    top = fmaxf(top, __shfl_xor_sync(~0u, top, 4));
                    top = fmaxf(top, __shfl_xor_sync(~0u, top, 8));
                    top = fmaxf(top, __shfl_xor_sync(~0u, top, 16));
                    const float now = fmaxf(m[nt][x], top);
                    // nothing seen yet: any finite reference will do, the weights are 0
                    const float ref = now == -INFINITY ? 0.0f : now;
                    alpha[nt][x] = pow2(m[nt][x] - ref);
                    m[nt][x] = now;
                    float sum = 0.0f;
#pragma unroll
                    for (int s = 0; s < TT; ++s)
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            float &v = sc[s][nt][2 * y + x];
                            v = pow2(v - ref + SHIFT);
                            sum += v;
                        }
                    l[nt][x] = fmaf(l[nt][x], alpha[nt][x], sum);
                }

            // ---- O = O alpha + V^T P^T ----
            // with `mixed`, for the query rows of the new token `row` alone, the values
            // behind its positions set to zero
            auto values = [&](auto mixed, int row) {
                constexpr bool MIXED = decltype(mixed)::value;
                const int n = len - R + row + 1;
                [[maybe_unused]] uint32_t keep[TT][2];  // of this thread's pairs of positions
                if constexpr (MIXED) {
#pragma unroll
                    for (int s = 0; s < TT; ++s)
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const int t = tile + 16 * s + 8 * y + 2 * c;
                            keep[s][y] = (t < n ? 0xffffu : 0u) | (t + 1 < n ? 0xffff0000u : 0u);
                        }
                }
                [[maybe_unused]] float unscale = 1.0f, vshrink = 1.0f;
                [[maybe_unused]] uint32_t vw[TT][2][SW];
                if constexpr (Q8) {
                    uint32_t top = 0;  // of the finite scales' bits: ordered as the numbers
#pragma unroll
                    for (int s = 0; s < TT; ++s)
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            scales_of(vs_s, s, y, vw[s][y]);
                            if (MIXED && tile + 16 * s + 8 * y + r >= n) {
#pragma unroll
                                for (int i = 0; i < SW; ++i) vw[s][y][i] = 0;
                            }
#pragma unroll
                            for (int i = 0; i < SW; ++i) {
                                const uint32_t lo = vw[s][y][i] & 0x7fffu, hi = vw[s][y][i] >> 16 & 0x7fffu;
                                if (lo < 0x7c00u) top = max(top, lo);
                                if (hi < 0x7c00u) top = max(top, hi);
                            }
                        }
                    top = __reduce_max_sync(~0u, top);
                    const int now = max(vexp, (int)(top >> 10) - 14);  // 2^now > top
                    vshrink = pow2((float)(vexp - now));
                    unscale = pow2((float)-now);
                    if constexpr (!MIXED) {
                        vexp = now;
                    } else {  // this warp's last tile
                        ended = true;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int x = 0; x < 2; ++x)
                                if (lim[nt][x] == n) vend[nt][x] = now;
                    }
                }
                uint32_t pf[TT][NT][PP][2];
                auto weights = [&](auto factor) {
#pragma unroll
                    for (int s = 0; s < TT; ++s)
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const float d = factor(s, y);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                float x0 = sc[s][nt][2 * y], x1 = sc[s][nt][2 * y + 1];
                                if constexpr (Q8) x0 *= d, x1 *= d;
                                const Words<PP> w = split_pair<HALF, PP>(x0, x1);
#pragma unroll
                                for (int p = 0; p < PP; ++p) pf[s][nt][p][y] = transpose8x8(w.w[p]);
                            }
                        }
                };
                if constexpr (!Q8) weights([](int, int) { return 1.0f; });
                [[maybe_unused]] uint2 vb[TT][4];
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    uint4 A[TT];
                    if constexpr (Q8) {
                        if (mt % 2 == 0) {
                            const int v = mt / 2;
                            weights([&](int s, int y) { return scale(vw[s][y], v) * unscale; });
#pragma unroll
                            for (int s = 0; s < TT; ++s)
#pragma unroll
                                for (int x = 0; x < 4; ++x) {
                                    const int in = 2 * c + (x & 1) + 8 * (x >> 1);
                                    const int key = (in & 7) & (ROWB / 16 - 1);
                                    const uint32_t w = *reinterpret_cast<const uint32_t *>(
                                        v_s + (16 * s + in) * ROWB + (((2 * v + (r >> 2)) ^ key) << 4) + 4 * (r & 3));
                                    vb[s][x] = codes_to_f16(w);
                                }
                        }
#pragma unroll
                        for (int s = 0; s < TT; ++s) {
                            uint32_t w[4];
#pragma unroll
                            for (int x = 0; x < 4; ++x) w[x] = mt % 2 ? vb[s][x].y : vb[s][x].x;
                            A[s] = make_uint4(__byte_perm(w[0], w[1], 0x5410), __byte_perm(w[0], w[1], 0x7632),
                                              __byte_perm(w[2], w[3], 0x5410), __byte_perm(w[2], w[3], 0x7632));
                        }
                    } else {
                        const int vrow = (lane & 7) + (lane >> 4) * 8;
#pragma unroll
                        for (int s = 0; s < TT; ++s)
                            A[s] = ldmatrix4_trans(smem_address(v_s) + (16 * s + vrow) * ROWB +
                                                   (((2 * mt + (lane >> 3 & 1)) ^ (vrow & 7)) << 4));
                    }
                    if constexpr (MIXED) {
#pragma unroll
                        for (int s = 0; s < TT; ++s) {
                            A[s].x &= keep[s][0], A[s].y &= keep[s][0];
                            A[s].z &= keep[s][1], A[s].w &= keep[s][1];
                        }
                    }
                    float t[NT][4];
#pragma unroll
                    for (int p = PP - 1; p >= 0; --p)
#pragma unroll
                        for (int s = 0; s < TT; ++s)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                if (p == PP - 1 && s == 0)
                                    mma16816<HALF, true>(t[nt], A[s], pf[s][nt][p][0], pf[s][nt][p][1]);
                                else
                                    mma16816<HALF>(t[nt], A[s], pf[s][nt][p][0], pf[s][nt][p][1]);
                            }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            if (!MIXED || lim[nt][x & 1] == n)
                                O[mt][nt][x] =
                                    fmaf(O[mt][nt][x], Q8 ? alpha[nt][x & 1] * vshrink : alpha[nt][x & 1], t[nt][x]);
                }
            };
            // A query row's own later positions carry weight 0, but 0 times a draft
            // token's NaN is NaN: a tile with positions that some rows do not see is
            // done token by token.  It is the last one of its warp: the new tokens lie
            // within two tiles, which belong to two warps.
            if (R > 1 && !shared && tile + TILE > len - R + 1) {
                for (int row = R - 1; row >= 0; --row) values(std::true_type{}, row);
            } else {
                values(std::false_type{}, 0);
            }
        }
        copies_wait<0>();
        __syncwarp();  // the ring is free: it takes this warp's O

        // ---- join of the four warps ----
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                float v = l[nt][x];
                v += __shfl_xor_sync(~0u, v, 4);
                v += __shfl_xor_sync(~0u, v, 8);
                v += __shfl_xor_sync(~0u, v, 16);
                if (r == 0) {
                    m_s[warp * ROWS + 8 * nt + 2 * c + x] = m[nt][x];
                    l_s[warp * ROWS + 8 * nt + 2 * c + x] = v;
                }
                const float back = Q8 ? pow2((float)(ended ? vend[nt][x] : vexp)) : 1.0f;
                float *dst = reinterpret_cast<float *>(ring) + (8 * nt + 2 * c + x) * S::OROW;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    const int d0 = Q8 ? 32 * (mt / 2) + 4 * r + 2 * (mt % 2) : 16 * mt + r;
                    dst[d0] = Q8 ? O[mt][nt][x] * back : O[mt][nt][x];
                    dst[d0 + (Q8 ? 1 : 8)] = Q8 ? O[mt][nt][x + 2] * back : O[mt][nt][x + 2];
                }
            }
        __syncthreads();
        const int chunks = attn_chunks(len, a.chunk);
        const long long unit = (((long long)b * a.max_chunks + ck) * KVH + h) * a.row_tiles + rt;
        for (int i = warp; i < ROWS; i += WARPS) {
            const int g = first_row + i;
            if (g >= group_rows) break;
            float top = m_s[i];
#pragma unroll
            for (int w = 1; w < WARPS; ++w) top = fmaxf(top, m_s[w * ROWS + i]);
            float sum = 0.0f, f[WARPS];
#pragma unroll
            for (int w = 0; w < WARPS; ++w) {
                const float mw = m_s[w * ROWS + i];
                f[w] = mw == -INFINITY ? 0.0f : pow2(mw - top);
                sum = fmaf(f[w], l_s[w * ROWS + i], sum);
            }
            auto joined = [&](int d) {
                float v = 0.0f;
#pragma unroll
                for (int w = 0; w < WARPS; ++w)
                    v = fmaf(f[w], reinterpret_cast<const float *>(smem + w * S::RING)[i * S::OROW + d], v);
                return v;
            };
            if (a.cluster) {  // this CTA's part of the join below, in warp 0's place
                for (int d = lane; d < D; d += 32) reinterpret_cast<float *>(smem)[i * S::OROW + d] = joined(d);
                __syncwarp();
                if (lane == 0) m_s[i] = top, l_s[i] = sum;
            } else if (chunks == 1 && !parts) {  // the result itself
                for (int d = lane; d < D; d += 32) attn_store(a, b, h, g, d, sum == 0.0f ? 0.0f : joined(d) / sum);
            } else {
                if (lane == 0) a.part_ml[unit * ROWS + i] = make_float2(top, sum);
                float *dst = a.part_o + (unit * ROWS + i) * D;
                for (int d = lane; d < D; d += 32) dst[d] = joined(d);
            }
        }
        if (a.cluster) {
            // ---- join of a request's chunks over the cluster's shared memory: each
            // CTA takes a share of the elements, chunk by chunk ----
            cluster_sync();
            const int n = a.max_chunks, all = min(ROWS, a.group_rows - first_row) * D;
            const uint32_t m_at = smem_address(m_s), l_at = smem_address(l_s), o_at = smem_address(smem);
            for (int e = ck * WARPS * 32 + tid; e < all; e += n * WARPS * 32) {
                const int i = e / D, d = e - i * D, g = first_row + i;
                float mk[ATTN_CLUSTER], top = -INFINITY;
#pragma unroll
                for (int k = 0; k < ATTN_CLUSTER; ++k) {
                    mk[k] = k < n ? peer_float(m_at + 4 * i, k) : -INFINITY;
                    top = fmaxf(top, mk[k]);
                }
                float sum = 0.0f, v = 0.0f;
#pragma unroll
                for (int k = 0; k < ATTN_CLUSTER; ++k)
                    if (k < n) {
                        const float f = mk[k] == -INFINITY ? 0.0f : pow2(mk[k] - top);
                        sum = fmaf(f, peer_float(l_at + 4 * i, k), sum);
                        v = fmaf(f, peer_float(o_at + 4 * (i * S::OROW + d), k), v);
                    }
                attn_store(a, b, h, g, d, sum == 0.0f ? 0.0f : v / sum);
            }
            cluster_sync();  // shared memory stays until the others have read it
        }
        __syncthreads();  // the next unit fills the rings and rewrites q_s and m_s
    }
}

template <int KV, int QP, int PP, int DP, int NT, bool MODES>
int attn_occupancy(size_t smem, int *out) {
    auto *kern = attn_kernel<KV, QP, PP, DP, NT, MODES>;
    static std::atomic<unsigned long long> known[64];  // per device: smem << 8 | CTAs per SM
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return (int)e;
    if (dev < 0 || dev >= 64) return (int)cudaErrorInvalidDevice;
    const unsigned long long was = known[dev].load();
    if (was >> 8 == smem) {
        *out = (int)(was & 255);
        return 0;
    }
    if (!was) {
        const int need = (int)(AttnShape<KV, QP, PP, DP, NT>::SMEM + (ATTN_MAX_REQUESTS + 1) * sizeof(int));
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, need);
        if (e != cudaSuccess) return (int)e;
    }
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(out, kern, ATTN_WARPS * 32, smem);
    if (e == cudaSuccess) known[dev].store((unsigned long long)smem << 8 | (unsigned)*out);
    return (int)e;
}

}  // namespace bq

// the instances of one cache type and way of carrying queries, for head_dim up to
// 64, 128 and 256, of the ordinary calls or (MODES) of those over shared pages
#define BQ_ATTN_INST(KV, QP, PP, DP, NT, MODES)                                                    \
    {                                                                                              \
        DP, NT, (size_t)bq::AttnShape<KV, QP, PP, DP, NT>::SMEM,                                   \
            bq::attn_occupancy<KV, QP, PP, DP, NT, MODES>,                                         \
            [](const bq::AttnArgs &a, int grid, size_t smem, void *stream,                         \
               unsigned int *status) -> cudaError_t {                                              \
                return bq::launch_pdl(bq::attn_kernel<KV, QP, PP, DP, NT, MODES>,                  \
                                      dim3((unsigned)grid), bq::ATTN_WARPS * 32, smem, stream,     \
                                      a.cluster ? a.max_chunks : 1, a, status);                    \
            }                                                                                      \
    }
#define BQ_ATTN_INSTS(KV, QP, PP, MODES)                                                           \
    BQ_ATTN_INST(KV, QP, PP, 64, 1, MODES), BQ_ATTN_INST(KV, QP, PP, 64, 2, MODES),                \
        BQ_ATTN_INST(KV, QP, PP, 128, 1, MODES), BQ_ATTN_INST(KV, QP, PP, 128, 2, MODES),          \
        BQ_ATTN_INST(KV, QP, PP, 256, 1, MODES), BQ_ATTN_INST(KV, QP, PP, 256, 2, MODES)
#define BQ_ATTN_UNIT(NAME, ...)                                                                    \
    const bq::AttnInstance *bq_internal_attn_##NAME(int *n) {                                      \
        static const bq::AttnInstance inst[] = {__VA_ARGS__};                                      \
        *n = (int)(sizeof inst / sizeof inst[0]);                                                  \
        return inst;                                                                               \
    }
