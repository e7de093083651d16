// bq_attn.cuh -- attention of a request's last one to six tokens over its paged
// key-value cache (bq_paged_attention in include/bqgemv.h).
//
// Mathematics.  Per query row: s_t = scale q.k_t, o = sum_t e^(s_t) v_t / sum_t e^(s_t)
// in one pass over the cache with a running maximum m and sum l: a tile with
// maximum m' rescales what was summed by 2^(m - m') (all exponents in base 2,
// the factor log2 e folded into scale).  The positions are cut into chunks of
// a fixed length, each chunk's tiles are shared by four warps, and the partial
// (m, l, O) are joined in a fixed order, by warps in shared memory and by
// chunks in a second kernel.  Which chunks exist depends on the geometry and
// the length alone, and an empty chunk joins with weight zero, so a row's bits
// depend on its own inputs and the geometry only.
//
// Bound by HBM: every live byte of the cache is read once (twice or more for
// the row tiles of more than 8 NT query rows per kv head, through L2), about
// 4 flop per byte and query row.  So the kernel is built around the loads:
//  - A warp loads 16-byte pieces of K and V rows from global memory straight
//    into the registers from which mma.sync reads them; no shared memory, no
//    barrier and no transposing copy stand between.  mma.sync sums over its
//    k index, so any order of the summed index will do as long as both
//    operands share it, and any order of the output rows:
//      S^T = K Q^T: rows are positions, summed over d.  Lane (r, c) = (lane /
//        4, lane % 4) takes d = 8 (c + 4 j) .. + 7 of positions r and r + 8:
//        one 16-byte load feeds two instructions.
//      O^T = V^T P^T: rows are d, summed over positions.  Lane (r, c) takes
//        d = 8 (r + 8 m) .. + 7 of positions 2c, 2c + 1, 2c + 8, 2c + 9; a
//        byte permute pairs two positions' values into an A register.
//    The scores come out with positions along r, the weights go in with
//    positions along c: movmatrix transposes the 8 x 8 tile in registers.
//  - The K registers of the next tile are loaded while the weights of this one
//    are computed, the V registers while its scores are.
//  - tcgen05 would hold 128 rows of accumulator for 1 to 48 query rows; with 8
//    query rows per n-tile the tensor pipe is about a fifth busy at HBM speed.
// Precision.  The tensor cores multiply 16-bit values exactly.  A query of
// the cache's own type is used as it is; any other is split into QP 16-bit
// parts (fp16: 2 parts, 22 bits, after scaling the row by a power of two; bf16:
// 3 parts, 24 bits), the weights into PP parts (2 for 16-bit queries, so that
// the output's own rounding stays the largest error).  Each tile's products
// are summed by the tensor core from zero, smallest parts first, and added to
// the fp32 accumulator by an fp32 FMA, since the tensor core truncates its sums.
// Q8_0 codes are exact in bf16; a key's scale multiplies its block's partial
// score, a value's scale its weight, both in fp32.
#pragma once

#include <cmath>

#include "bq_attn.h"

namespace bq {

enum { KV_F16 = 0, KV_BF16 = 1, KV_Q8 = 2 };

template <int N>
struct Words {
    uint32_t w[N];
};

__device__ __forceinline__ uint4 ldg16(const void *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}
__device__ __forceinline__ uint2 ldg8(const void *p) {
    uint2 v;
    asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}
__device__ __forceinline__ uint32_t ldg4(const void *p) {
    uint32_t v;
    asm volatile("ld.global.L1::no_allocate.u32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}

template <bool HALF>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (HALF)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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

// four int8 codes as two pairs of bf16.  With b = code mod 256 and the
// exponent byte 0x43, 0x4300 | (b & 127) is 128 + (b & 127) and 0x4300 | (b &
// 128) is 128 or 256, both whole numbers that bf16 holds; their difference is
// the code, exact.
__device__ __forceinline__ uint2 codes_to_bf16(uint32_t w) {
    uint2 o;
    const uint32_t lo = __byte_perm(w, 0x43434343u, 0x4140), hi = __byte_perm(w, 0x43434343u, 0x4342);
    const uint32_t la = lo & 0xff7fff7fu, lb = lo & 0xff80ff80u;
    const uint32_t ha = hi & 0xff7fff7fu, hb = hi & 0xff80ff80u;
    asm("sub.bf16x2 %0, %1, %2;" : "=r"(o.x) : "r"(la), "r"(lb));
    asm("sub.bf16x2 %0, %1, %2;" : "=r"(o.y) : "r"(ha), "r"(hb));
    return o;
}

template <int KV, int QP, int PP, int DP, int NT>
struct AttnShape {
    static constexpr bool Q8 = KV == KV_Q8, HALF = KV == KV_F16;
    static constexpr int ROWS = 8 * NT;
    // positions per tile and warp, in steps of 16: enough loads in flight for
    // the registers at hand
    static constexpr int TT = Q8 ? (DP <= 128 ? 2 : 1) : (DP <= 64 ? 2 : 1);
    static constexpr int QROW = 2 * DP + 64;  // bytes: rows 64 apart modulo 128, so 8 lanes' 16-byte
                                              // reads of 2 rows and 4 pieces hit 8 bank groups
    static constexpr int Q_BYTES = QP * ROWS * QROW;
    static constexpr int O_BYTES = ATTN_WARPS * ROWS * DP * 4;
    // q parts, the join of the warps, row statistics
    static constexpr int SMEM = Q_BYTES + O_BYTES + (2 * ATTN_WARPS + 1) * ROWS * 4;
    // resident CTAs that the registers are sized for
    static constexpr int OCC = DP * NT <= 64 ? 4 : DP * NT <= 128 ? 3 : 2;
};

template <int KV, int QP, int PP, int DP, int NT>
__global__ void __launch_bounds__(ATTN_WARPS * 32, AttnShape<KV, QP, PP, DP, NT>::OCC)
    attn_kernel(const __grid_constant__ AttnArgs a, unsigned int *status) {
    using S = AttnShape<KV, QP, PP, DP, NT>;
    constexpr bool Q8 = S::Q8, HALF = S::HALF;
    constexpr int TT = S::TT, ROWS = S::ROWS, TILE = 16 * TT;
    constexpr int KJ = DP / 32;             // groups of 32 d per row in S^T
    constexpr int KW = Q8 ? 2 : 4;          // words of a K piece (8 values)
    constexpr int VM = Q8 ? DP / 32 : DP / 64;  // pieces per position in O^T
    constexpr int VW = Q8 ? 1 : 4;          // words of a V piece
    constexpr int OJ = Q8 ? 2 : 4;          // 16-row output tiles per piece
    constexpr float SHIFT = HALF ? (float)ATTN_SHIFT_F16 : 0.0f;
    extern __shared__ __align__(16) uint8_t smem[];
    uint8_t *q_s = smem;
    float *o_s = reinterpret_cast<float *>(smem + S::Q_BYTES);
    float *m_s = o_s + ATTN_WARPS * ROWS * DP, *l_s = m_s + ATTN_WARPS * ROWS;
    float *f_s = l_s + ATTN_WARPS * ROWS;          // per row: factor of its scores
    int *pre = reinterpret_cast<int *>(f_s + ROWS);  // [requests + 1]
    __shared__ int scan_s[ATTN_WARPS];

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = lane >> 2, c = lane & 3;
    const int B = a.x.requests, R = a.x.rows, D = a.c.head_dim, KVH = a.c.kv_heads;
    const int most = a.x.table_width * a.c.page_size;
    pdl_wait();
    if (a.max_chunks > 1) pdl_launch_dependents();

    auto length = [&](int b) { return min(max(a.x.lens[b], 0), most); };
    // exclusive prefix sums of the requests' units
    {
        const int per = (B + ATTN_WARPS * 32 - 1) / (ATTN_WARPS * 32);
        const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
        int n = 0;
        for (int b = b0; b < b1; ++b) {
            const int len = a.x.lens[b];
            if ((len < 0 || len > most) && blockIdx.x == 0) atomicOr(status, BQ_DEVERR_LENGTH);
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
    const long long per_chunk = (long long)KVH * a.row_tiles;
    const long long units = pre[B] * per_chunk;

    for (long long u = blockIdx.x; u < units; u += gridDim.x) {
        const int cu = (int)(u / per_chunk), hr = (int)(u - cu * per_chunk);
        const int h = hr / a.row_tiles, rt = hr - h * a.row_tiles;
        int b = 0;
        for (int hi = B; hi - b > 1;) {
            const int mid = (b + hi) >> 1;
            if (pre[mid] <= cu) b = mid;
            else hi = mid;
        }
        const int ck = cu - pre[b], len = length(b);
        const int begin = ck * a.chunk, end = min(len, begin + a.chunk);
        const int first_row = rt * ROWS;

        // ---- queries: fp32 -> 16-bit parts in shared memory ----
        for (int i = warp; i < ROWS; i += ATTN_WARPS) {
            const int g = first_row + i;
            float x[DP / 32];
            float top = 0.0f;
            if (g < a.group_rows) {
                const int row = (int)a.group.div((uint32_t)g);
                const int head = h * (int)a.group.d + g - row * (int)a.group.d;
                const long long at = ((long long)b * R + row) * a.x.q_row_stride + head * a.x.q_head_stride;
#pragma unroll
                for (int e = 0; e < DP / 32; ++e) {
                    const int d = lane + 32 * e;
                    x[e] = d >= D ? 0.0f
                           : a.x.dtype == BQ_F32 ? ((const float *)a.x.q)[at + d]
                           : a.x.dtype == BQ_F16 ? __half2float(((const __half *)a.x.q)[at + d])
                                                 : __bfloat162float(((const __nv_bfloat16 *)a.x.q)[at + d]);
                    top = fmaxf(top, fabsf(x[e]));
                }
            } else {
#pragma unroll
                for (int e = 0; e < DP / 32; ++e) x[e] = 0.0f;
            }
            float factor = a.scale_log2;
            if constexpr (HALF && QP > 1) {
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
                lim[nt][x] = g < a.group_rows ? len - R + (int)a.group.div((uint32_t)g) + 1 : 0;
                fac[nt][x] = f_s[i];
            }

        float O[VM][OJ][NT][4], m[NT][2], l[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt][0] = m[nt][1] = -INFINITY;
            l[nt][0] = l[nt][1] = 0.0f;
#pragma unroll
            for (int v = 0; v < VM; ++v)
#pragma unroll
                for (int j = 0; j < OJ; ++j)
#pragma unroll
                    for (int x = 0; x < 4; ++x) O[v][j][nt][x] = 0.0f;
        }

        const int *row_table = a.x.table + b * a.x.table_stride;
        const long long head_off = (long long)h * a.c.head_stride;
        // element offset of this lane's position of a tile, -1 where there is none
        auto entry_of = [&](int t) { return t < end ? row_table[a.page.div((uint32_t)t)] : -1; };
        auto offset_of = [&](int t, int page) -> long long {
            if (t >= end) return -1;
            if (page < 0 || page >= a.c.pages) {
                atomicOr(status, BQ_DEVERR_PAGE);
                return -1;
            }
            const uint32_t in_page = (uint32_t)t - a.page.div((uint32_t)t) * a.page.d;
            return page * a.c.page_stride + in_page * a.c.slot_stride + head_off;
        };
        uint32_t kreg[TT][2][KJ][KW];
        [[maybe_unused]] __half kscale[TT][2][KJ];
        auto load_k = [&](long long off) {
#pragma unroll
            for (int s = 0; s < TT; ++s)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const long long o = __shfl_sync(~0u, off, 16 * s + 8 * x + r);
#pragma unroll
                    for (int j = 0; j < KJ; ++j) {
                        const bool ok = o >= 0 && 8 * (c + 4 * j) < D;
                        if constexpr (Q8) {
                            const uint2 v = ok ? ldg8((const uint8_t *)a.c.k + o + 8 * (c + 4 * j)) : make_uint2(0, 0);
                            kreg[s][x][j][0] = v.x, kreg[s][x][j][1] = v.y;
                            kscale[s][x][j] = ok ? ((const __half *)a.c.k_scale)[(o >> 5) + j] : __half(0.0f);
                        } else {
                            const uint4 v = ok ? ldg16((const uint8_t *)a.c.k + 2 * o + 16 * (c + 4 * j))
                                               : make_uint4(0, 0, 0, 0);
                            kreg[s][x][j][0] = v.x, kreg[s][x][j][1] = v.y;
                            kreg[s][x][j][KW - 2] = v.z, kreg[s][x][j][KW - 1] = v.w;
                        }
                    }
                }
        };

        int tile = begin + warp * TILE;
        const int stride = ATTN_WARPS * TILE;
        const int mine = lane & (TILE - 1);
        int entry = entry_of(tile + mine);
        long long off = offset_of(tile + mine, entry);
        if (tile < end) load_k(off);
        entry = entry_of(tile + stride + mine);

        for (; tile < end; tile += stride) {
            // ---- V of this tile on its way while the scores are computed ----
            uint32_t vreg[TT][4][VM][VW];
            [[maybe_unused]] __half vscale[TT][2][VM];
#pragma unroll
            for (int s = 0; s < TT; ++s) {
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const long long o = __shfl_sync(~0u, off, 16 * s + 2 * c + (x & 1) + 8 * (x >> 1));
#pragma unroll
                    for (int v = 0; v < VM; ++v) {
                        if constexpr (Q8) {
                            const bool ok = o >= 0 && 32 * v < D;
                            vreg[s][x][v][0] = ok ? ldg4((const uint8_t *)a.c.v + o + 32 * v + 4 * r) : 0;
                        } else {
                            const bool ok = o >= 0 && 8 * (r + 8 * v) < D;
                            const uint4 w = ok ? ldg16((const uint8_t *)a.c.v + 2 * o + 16 * (r + 8 * v))
                                               : make_uint4(0, 0, 0, 0);
                            vreg[s][x][v][0] = w.x, vreg[s][x][v][VW > 1 ? 1 : 0] = w.y;
                            vreg[s][x][v][VW > 2 ? 2 : 0] = w.z, vreg[s][x][v][VW > 3 ? 3 : 0] = w.w;
                        }
                    }
                }
                if constexpr (Q8) {
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const long long o = __shfl_sync(~0u, off, 16 * s + 8 * x + r);
#pragma unroll
                        for (int v = 0; v < VM; ++v)
                            vscale[s][x][v] =
                                o >= 0 && 32 * v < D ? ((const __half *)a.c.v_scale)[(o >> 5) + v] : __half(0.0f);
                    }
                }
            }
            // masked as bad pages are: positions whose offset is -1
            bool live[TT][2];
#pragma unroll
            for (int s = 0; s < TT; ++s)
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    live[s][x] = __shfl_sync(~0u, (int)(off >= 0), 16 * s + 8 * x + r) != 0;

            // ---- scores ----
            float sc[TT][NT][4];
#pragma unroll
            for (int s = 0; s < TT; ++s)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int x = 0; x < 4; ++x) sc[s][nt][x] = 0.0f;
            if constexpr (Q8) {
#pragma unroll
                for (int j = 0; j < KJ; ++j) {
                    uint2 k0[TT][2], k1[TT][2];  // [pieces' first and second 4 codes]
#pragma unroll
                    for (int s = 0; s < TT; ++s)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            k0[s][x] = codes_to_bf16(kreg[s][x][j][0]);
                            k1[s][x] = codes_to_bf16(kreg[s][x][j][1]);
                        }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float t[TT][4];
#pragma unroll
                        for (int s = 0; s < TT; ++s) t[s][0] = t[s][1] = t[s][2] = t[s][3] = 0.0f;
#pragma unroll
                        for (int p = QP - 1; p >= 0; --p) {
                            const uint4 q = *reinterpret_cast<const uint4 *>(
                                q_s + (p * ROWS + 8 * nt + r) * S::QROW + 16 * (c + 4 * j));
#pragma unroll
                            for (int s = 0; s < TT; ++s) {
                                mma16816<HALF>(t[s], k0[s][0].x, k0[s][1].x, k0[s][0].y, k0[s][1].y, q.x, q.y);
                                mma16816<HALF>(t[s], k1[s][0].x, k1[s][1].x, k1[s][0].y, k1[s][1].y, q.z, q.w);
                            }
                        }
#pragma unroll
                        for (int s = 0; s < TT; ++s) {
                            const float d0 = __half2float(kscale[s][0][j]), d1 = __half2float(kscale[s][1][j]);
                            sc[s][nt][0] = fmaf(d0, t[s][0], sc[s][nt][0]);
                            sc[s][nt][1] = fmaf(d0, t[s][1], sc[s][nt][1]);
                            sc[s][nt][2] = fmaf(d1, t[s][2], sc[s][nt][2]);
                            sc[s][nt][3] = fmaf(d1, t[s][3], sc[s][nt][3]);
                        }
                    }
                }
            } else {
#pragma unroll
                for (int p = QP - 1; p >= 0; --p)
#pragma unroll
                    for (int j = 0; j < KJ; ++j)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const uint4 q = *reinterpret_cast<const uint4 *>(
                                q_s + (p * ROWS + 8 * nt + r) * S::QROW + 16 * (c + 4 * j));
#pragma unroll
                            for (int s = 0; s < TT; ++s) {
                                mma16816<HALF>(sc[s][nt], kreg[s][0][j][0], kreg[s][1][j][0], kreg[s][0][j][1],
                                               kreg[s][1][j][1], q.x, q.y);
                                mma16816<HALF>(sc[s][nt], kreg[s][0][j][KW - 2], kreg[s][1][j][KW - 2],
                                               kreg[s][0][j][KW - 1], kreg[s][1][j][KW - 1], q.z, q.w);
                            }
                        }
            }

            // ---- K of the next tile, table entry of the one after it ----
            const int next = tile + stride;
            off = offset_of(next + mine, entry);
            if (next < end) load_k(off);
            entry = entry_of(next + stride + mine);

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
                            v = t < lim[nt][x] && live[s][y] ? v * fac[nt][x] : -INFINITY;
                            top = fmaxf(top, v);
                        }
                    top = fmaxf(top, __shfl_xor_sync(~0u, top, 4));
                    top = fmaxf(top, __shfl_xor_sync(~0u, top, 8));
                    top = fmaxf(top, __shfl_xor_sync(~0u, top, 16));
                    const float now = fmaxf(m[nt][x], top);
                    // nothing seen yet: any finite reference will do, the weights are 0
                    const float ref = now == -INFINITY ? 0.0f : now;
                    alpha[nt][x] = exp2f(m[nt][x] - ref);
                    m[nt][x] = now;
                    float sum = 0.0f;
#pragma unroll
                    for (int s = 0; s < TT; ++s)
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            float &v = sc[s][nt][2 * y + x];
                            v = exp2f(v - ref + SHIFT);
                            sum += v;
                        }
                    l[nt][x] = fmaf(l[nt][x], alpha[nt][x], sum);
                }

            // ---- O = O alpha + V^T P^T.  A query row's own later positions carry
            // weight 0, but 0 times a draft token's NaN is NaN: a tile that holds
            // positions some rows do not see is done row by row, last row first, the
            // values behind the row's positions set to zero ----
            const bool mixed = R > 1 && tile + TILE > len - R + 1;
            const int passes = mixed ? R : 1;
            for (int pass = 0; pass < passes; ++pass) {
                const int row = R - 1 - pass;
                bool take[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int x = 0; x < 2; ++x) take[nt][x] = !mixed || lim[nt][x] == len - R + row + 1;
                if (mixed) {
                    const int n = len - R + row + 1;
#pragma unroll
                    for (int s = 0; s < TT; ++s)
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            if (tile + 16 * s + 2 * c + (x & 1) + 8 * (x >> 1) >= n)
#pragma unroll
                                for (int v = 0; v < VM; ++v)
#pragma unroll
                                    for (int w = 0; w < VW; ++w) vreg[s][x][v][w] = 0;
                }
                uint32_t pf[TT][NT][PP][2];
                if constexpr (!Q8) {
#pragma unroll
                    for (int s = 0; s < TT; ++s)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                const Words<PP> w = split_pair<HALF, PP>(sc[s][nt][2 * y], sc[s][nt][2 * y + 1]);
#pragma unroll
                                for (int p = 0; p < PP; ++p) pf[s][nt][p][y] = transpose8x8(w.w[p]);
                            }
                }
#pragma unroll
                for (int v = 0; v < VM; ++v) {
                    if constexpr (Q8) {
#pragma unroll
                        for (int s = 0; s < TT; ++s)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int y = 0; y < 2; ++y) {
                                    const float d = __half2float(vscale[s][y][v]);
                                    const Words<PP> w =
                                        split_pair<HALF, PP>(sc[s][nt][2 * y] * d, sc[s][nt][2 * y + 1] * d);
#pragma unroll
                                    for (int p = 0; p < PP; ++p) pf[s][nt][p][y] = transpose8x8(w.w[p]);
                                }
                    }
                    [[maybe_unused]] uint2 vb[TT][4];
                    if constexpr (Q8) {
#pragma unroll
                        for (int s = 0; s < TT; ++s)
#pragma unroll
                            for (int x = 0; x < 4; ++x) vb[s][x] = codes_to_bf16(vreg[s][x][v][0]);
                    }
#pragma unroll
                    for (int j = 0; j < OJ; ++j) {
                        float t[NT][4];
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) t[nt][0] = t[nt][1] = t[nt][2] = t[nt][3] = 0.0f;
                        uint32_t A[TT][4];
#pragma unroll
                        for (int s = 0; s < TT; ++s) {
                            uint32_t w[4];
#pragma unroll
                            for (int x = 0; x < 4; ++x) {
                                if constexpr (Q8) w[x] = j ? vb[s][x].y : vb[s][x].x;
                                else w[x] = vreg[s][x][v][j];
                            }
                            A[s][0] = __byte_perm(w[0], w[1], 0x5410);
                            A[s][1] = __byte_perm(w[0], w[1], 0x7632);
                            A[s][2] = __byte_perm(w[2], w[3], 0x5410);
                            A[s][3] = __byte_perm(w[2], w[3], 0x7632);
                        }
#pragma unroll
                        for (int p = PP - 1; p >= 0; --p)
#pragma unroll
                            for (int s = 0; s < TT; ++s)
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
                                    mma16816<HALF>(t[nt], A[s][0], A[s][1], A[s][2], A[s][3], pf[s][nt][p][0],
                                                   pf[s][nt][p][1]);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int x = 0; x < 4; ++x) {
                                float &o = O[v][j][nt][x];
                                if (take[nt][x & 1]) o = fmaf(o, alpha[nt][x & 1], t[nt][x]);
                            }
                    }
                }
            }
        }

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
            }
        __syncthreads();
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int i = 8 * nt + 2 * c + x;
                float top = m_s[i];
#pragma unroll
                for (int w = 1; w < ATTN_WARPS; ++w) top = fmaxf(top, m_s[w * ROWS + i]);
                const float f = m[nt][x] == -INFINITY ? 0.0f : exp2f(m[nt][x] - top);
                float *dst = o_s + (warp * ROWS + i) * DP;
#pragma unroll
                for (int v = 0; v < VM; ++v) {
                    // this thread's values of d: 2 OJ consecutive ones
                    float *at = dst + (Q8 ? 32 * v + 4 * r : 8 * (r + 8 * v));
#pragma unroll
                    for (int j = 0; j < OJ; ++j) {
                        at[2 * j] = O[v][j][nt][x] * f;
                        at[2 * j + 1] = O[v][j][nt][x + 2] * f;
                    }
                }
            }
        __syncthreads();
        const bool whole = pre[b + 1] - pre[b] == 1;  // one unit: the result itself
        const long long unit = (((long long)b * a.max_chunks + ck) * KVH + h) * a.row_tiles + rt;
        for (int i = warp; i < ROWS; i += ATTN_WARPS) {
            const int g = first_row + i;
            if (g >= a.group_rows) break;
            float top = m_s[i];
#pragma unroll
            for (int w = 1; w < ATTN_WARPS; ++w) top = fmaxf(top, m_s[w * ROWS + i]);
            float sum = 0.0f;
#pragma unroll
            for (int w = 0; w < ATTN_WARPS; ++w) {
                const float mw = m_s[w * ROWS + i];
                sum += mw == -INFINITY ? 0.0f : l_s[w * ROWS + i] * exp2f(mw - top);
            }
            const int row = (int)a.group.div((uint32_t)g);
            if (whole) {
                const int head = h * (int)a.group.d + g - row * (int)a.group.d;
                const long long at = ((long long)b * R + row) * a.x.out_row_stride + head * a.x.out_head_stride;
                const bool empty = len - R + row + 1 <= 0;
                for (int d = lane; d < D; d += 32) {
                    float v = 0.0f;
#pragma unroll
                    for (int w = 0; w < ATTN_WARPS; ++w) v += o_s[(w * ROWS + i) * DP + d];
                    v = empty ? 0.0f : v / sum;
                    if (a.x.dtype == BQ_F32) ((float *)a.x.out)[at + d] = v;
                    else if (a.x.dtype == BQ_F16) ((__half *)a.x.out)[at + d] = __float2half_rn(v);
                    else ((__nv_bfloat16 *)a.x.out)[at + d] = __float2bfloat16_rn(v);
                }
            } else {
                if (lane == 0) a.part_ml[unit * ROWS + i] = make_float2(top, sum);
                float *dst = a.part_o + (unit * ROWS + i) * D;
                for (int d = lane; d < D; d += 32) {
                    float v = 0.0f;
#pragma unroll
                    for (int w = 0; w < ATTN_WARPS; ++w) v += o_s[(w * ROWS + i) * DP + d];
                    dst[d] = v;
                }
            }
        }
        __syncthreads();  // the next unit rewrites q_s, m_s and o_s
    }
}

template <int KV, int QP, int PP, int DP, int NT>
int attn_occupancy(size_t smem, int *out) {
    auto *kern = attn_kernel<KV, QP, PP, DP, NT>;
    static std::atomic<int> set[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return (int)e;
    if (dev < 0 || dev >= 64) return (int)cudaErrorInvalidDevice;
    const int need = (int)(AttnShape<KV, QP, PP, DP, NT>::SMEM + (ATTN_MAX_REQUESTS + 1) * sizeof(int));
    if (!set[dev].load()) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, need);
        if (e != cudaSuccess) return (int)e;
        set[dev].store(1);
    }
    return (int)cudaOccupancyMaxActiveBlocksPerMultiprocessor(out, kern, ATTN_WARPS * 32, smem);
}

}  // namespace bq

// the instances of one cache type: parts 1 (q in the cache's 16-bit type) and
// the split one, for head_dim up to 64, 128 and 256
#define BQ_ATTN_INST(NAME, KV, PARTS, QP, PP, DP, NT)                                              \
    {                                                                                              \
        KV, PARTS, DP, NT, bq::ATTN_WARPS * 32, (size_t)bq::AttnShape<KV, QP, PP, DP, NT>::SMEM,   \
            bq::attn_occupancy<KV, QP, PP, DP, NT>,                                                \
            [](const bq::AttnArgs &a, int grid, size_t smem, void *stream) -> cudaError_t {        \
                unsigned int *status = nullptr;                                                    \
                cudaError_t e = status_addr_##NAME(&status);                                       \
                if (e != cudaSuccess) return e;                                                    \
                return bq::launch_pdl(bq::attn_kernel<KV, QP, PP, DP, NT>, dim3((unsigned)grid),   \
                                      bq::ATTN_WARPS * 32, smem, stream, 1, a, status);            \
            }                                                                                      \
    }
#define BQ_ATTN_UNIT(NAME, KV, QP1, PP1, QPS, PPS)                                                 \
    BQ_STATUS_WORD(attn_##NAME)                                                                    \
    static cudaError_t status_addr_##NAME(unsigned int **out) {                                    \
        static std::atomic<unsigned int *> addr[64];                                               \
        int dev = 0;                                                                               \
        cudaError_t e = cudaGetDevice(&dev);                                                       \
        if (e != cudaSuccess) return e;                                                            \
        if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;                                   \
        unsigned int *p = addr[dev].load();                                                        \
        if (!p) {                                                                                  \
            e = cudaGetSymbolAddress(reinterpret_cast<void **>(&p), g_status_attn_##NAME);         \
            if (e != cudaSuccess) return e;                                                        \
            addr[dev].store(p);                                                                    \
        }                                                                                          \
        *out = p;                                                                                  \
        return cudaSuccess;                                                                        \
    }                                                                                              \
    const bq::AttnInstance *bq_internal_attn_##NAME(int *n) {                                      \
        static const bq::AttnInstance inst[] = {                                                   \
            BQ_ATTN_INST(NAME, KV, 1, QP1, PP1, 64, 1),  BQ_ATTN_INST(NAME, KV, 1, QP1, PP1, 64, 2),   \
            BQ_ATTN_INST(NAME, KV, 1, QP1, PP1, 128, 1), BQ_ATTN_INST(NAME, KV, 1, QP1, PP1, 128, 2),  \
            BQ_ATTN_INST(NAME, KV, 1, QP1, PP1, 256, 1), BQ_ATTN_INST(NAME, KV, 2, QPS, PPS, 64, 1),   \
            BQ_ATTN_INST(NAME, KV, 2, QPS, PPS, 64, 2),  BQ_ATTN_INST(NAME, KV, 2, QPS, PPS, 128, 1),  \
            BQ_ATTN_INST(NAME, KV, 2, QPS, PPS, 128, 2), BQ_ATTN_INST(NAME, KV, 2, QPS, PPS, 256, 1)}; \
        *n = (int)(sizeof inst / sizeof inst[0]);                                                  \
        return inst;                                                                               \
    }                                                                                              \
    int bq_internal_attn_status_##NAME(unsigned int *flags, int clear) {                           \
        return read_status_attn_##NAME(flags, clear);                                              \
    }
