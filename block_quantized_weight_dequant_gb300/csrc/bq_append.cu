// bq_append.cu -- keys and values of new tokens into the paged cache, with
// rotary positions of one to three axes (bq_kv_append in include/bqgemv.h).
//
// Angles: the turn of pair p at position n is n * freq / (2 pi).  freq/(2 pi)
// is split once per thread into hi + lo (two fp32 words, 48 bits); per token
// n * hi is formed exactly as product and remainder (one FMUL, one FFMA), each
// reduced by its nearest whole number, and beyond 2^24, where n has a remainder
// of its own, so are the products with it and with lo.  So the fraction of a turn is
// right to about 2^-23 of a turn plus n * freq * 2^-50, at positions up to 2^31.  fp64
// runs once per thread and pair only (its rate is far below fp32's).
//
// A CTA takes a few tokens at a time: its threads put the tokens' cosines and
// sines into shared memory, one pair each, then its warps turn and store the
// tokens' heads.  A lane keeps to the same heads for all tokens, so that their
// addresses are one multiply-add a token, and copies its own values of the next
// MAX_BATCH tokens into its own place in shared memory (cp.async, no barrier).
// A lane holds 8 values of a head, so that a warp takes 1, 2 or 4 heads: the
// two quarters 4i .. 4i+3 and rot/2 + 4i .. of four (p, p + rot/2) pairs, or 8
// values in a row (four interleaved pairs, or values behind rot).  So no value
// moves between lanes for the rotation; a Q8_0 block is the first (or second)
// quarter of 8 lanes, or both of 4, or, where rot / 2 is not whole blocks, is
// put in order through shared memory.
//
// Bound by HBM for a prompt, by latency for one token.  Measured: 8192 tokens of
// 28 + 4 + 4 heads of 128, fp32 into fp16: 50 us, 5.7 TB/s; into Q8_0 48 us, 5.8
// TB/s; 4001 tokens of 16 + 4 + 4, bf16: 13 us; one token: 2.8 us.
#include <atomic>
#include <cmath>
#include <type_traits>

#include "bq_cache.cuh"

namespace {

BQ_STATUS_WORD(append)

constexpr int MAX_WARPS = 12;  // of a CTA: as many as a token's heads need
constexpr int MAX_BATCH = 4;  // tokens at a time
constexpr int UNROLL = 2;     // times the heads of a warp that it takes of a token

struct Args {
    bq_kv_cache c;
    bq_kv_append_args x;
    bq::FastDiv page;
    int items;  // heads of a token: q, k and v
    int parts;  // CTAs that share a token's heads
    int warps;  // of a CTA
    int batch;  // tokens at a time
    int smem;   // of a CTA, beside the static
    int wide, wide_out;  // 4-element accesses of the inputs, of q_out
    // strides (below 2^31) as 32-bit numbers: a product with an index is one instruction
    uint32_t q_t, q_h, k_t, k_h, v_t, v_h, o_t, o_h, page_s, head_s, slot_s;
};

// The Q8_0 code of x in its low byte: clamp(round(x / d), -127, 127), the fp32
// quotient rounded to nearest and then half away from zero, without the division.
// Any half h = c - 1/2 has at most 8 bits and d, an fp16 number, 11, so h d is an
// fp32 number; the fp32 numbers below it are below it by 2^-24 of it or more, and
// so are their quotients below h, which therefore round to less than h.  So the
// quotient's rounding does not matter: the code is the largest c with |x| >= (c -
// 1/2) d.  The guess, |x| / d taken a little small (`inv` is 1 / d less 2^-21 of it or
// more) and rounded to nearest, is that c or one less.  rest = |x| - guess d is
// exact: at most d in magnitude and a multiple of |x|'s last place or of d's, so
// rest >= d / 2 decides.  A NaN ends at -127, as in bq_quantize_pack.  d is not 0.
__device__ __forceinline__ uint32_t q8_code(float x, float d, float half_d, float inv) {
    constexpr float WHOLE = 12582912.0f;  // 1.5 2^23: added, the low bits are the whole number
    const float v = fabsf(x);
    float c = __fadd_rn(__fmaf_rn(v, inv, WHOLE), -WHOLE);
    if (__fmaf_rn(-c, d, v) >= half_d) c += 1.0f;
    c = fminf(fmaxf(copysignf(c, x), -127.0f), 127.0f);
    return __float_as_uint(c + WHOLE);
}

// 4 elements to shared memory, asynchronously
template <class T>
__device__ __forceinline__ void copy4(void *dst, const T *src) {
    const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
    if constexpr (sizeof(T) == 4)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(src) : "memory");
}

// GL lanes per head: 8 for head_dim up to 64, 16 up to 128, 32 up to 256
template <class E, int CT, int GL>
__global__ void __launch_bounds__(MAX_WARPS * 32, 2) append_kernel(const __grid_constant__ Args a) {
    using T = typename E::T;
    constexpr int HPW = 32 / GL;       // heads of a warp at a time
    constexpr int HALF_MAX = 4 * GL;   // pairs of a head
    constexpr int DMAX = 8 * GL;
    __shared__ __align__(16) float2 cs_s[2][MAX_BATCH][HALF_MAX];
    __shared__ long long row_s[2][MAX_BATCH];
    // [MAX_BATCH][UNROLL][2][threads] vectors, then the heads of each warp at a time
    // where Q8_0 blocks are put in order
    extern __shared__ __align__(16) uint8_t ahead_s[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int sub = lane / GL, i = lane % GL;
    const int part = blockIdx.x % a.parts;
    const long long groups = gridDim.x / a.parts;
    const int D = a.c.head_dim, rot = a.x.freq ? a.x.rot : 0, half = rot >> 1;
    const int WARPS = blockDim.x >> 5;
    bq::pdl_wait();

    const int heads = a.x.q ? a.x.heads : 0, kv = a.c.kv_heads;
    const long long slots_all = a.c.pages * a.c.page_size;
    const bool in_rot = 8 * i < rot, apart = in_rot && !a.x.interleaved;
    const int e0 = apart ? 4 * i : 8 * i, e1 = apart ? half + 4 * i : 8 * i + 4;
    const bool there = 8 * i < D;
    // The heads of every token that this lane takes, and where they come from and
    // go to: the same for all tokens, so that an address is one multiply-add.
    int type[UNROLL];          // 0 query, 1 key, 2 value, 3 none
    const T *src[UNROLL];      // of token 0
    uint32_t src_step[UNROLL];
    T *out[UNROLL];            // of a query of token 0
    uint32_t head_at[UNROLL];  // of a key's or value's head in its page
    bool any_kept[UNROLL];     // a key or value among this warp's heads
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
        const int item = ((part * UNROLL + u) * WARPS + warp) * HPW + sub;
        type[u] = item >= a.items ? 3 : item < heads ? 0 : item < heads + kv ? 1 : 2;
        const uint32_t head = item - (type[u] == 1 ? heads : type[u] == 2 ? heads + kv : 0);
        src[u] = type[u] == 0   ? (const T *)a.x.q + (uint64_t)head * a.q_h
                 : type[u] == 1 ? (const T *)a.x.k + (uint64_t)head * a.k_h
                                : (const T *)a.x.v + (uint64_t)head * a.v_h;
        src_step[u] = type[u] == 0 ? a.q_t : type[u] == 1 ? a.k_t : a.v_t;
        out[u] = type[u] == 0 ? (T *)a.x.q_out + (uint64_t)head * a.o_h : nullptr;
        head_at[u] = head;
        if (!there && CT != BQ_Q8_0) type[u] = 3;
        any_kept[u] = __any_sync(~0u, type[u] == 1 || type[u] == 2);
    }

    // This lane's values of a token on their way into its own place in shared
    // memory, MAX_BATCH tokens ahead (rows that allow no wide access are read when
    // they are used).
    constexpr int VEC = 4 * (int)sizeof(T);
    float *order_s = reinterpret_cast<float *>(ahead_s + MAX_BATCH * UNROLL * 2 * (int)blockDim.x * VEC);
    auto place = [&](int b, int u, int v) { return ahead_s + ((b * UNROLL + u) * 2 + v) * (int)blockDim.x * VEC + tid * VEC; };
    auto fetch = [&](long long t, int b) {
        if (a.wide && t < a.x.tokens) {
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {
                if (type[u] == 3 || !there) continue;
                const T *at = src[u] + (uint64_t)(uint32_t)t * src_step[u];
                copy4(place(b, u, 0), at + e0);
                copy4(place(b, u, 1), at + e1);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto load = [&](uint32_t t, int b, float (&x)[UNROLL][2][4]) {
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            if (type[u] == 3 || !there) continue;
            if (a.wide) {
                bq::load_wide<E, 4>(reinterpret_cast<const T *>(place(b, u, 0)), x[u][0]);
                bq::load_wide<E, 4>(reinterpret_cast<const T *>(place(b, u, 1)), x[u][1]);
            } else {
                const T *at = src[u] + (uint64_t)t * src_step[u];
                bq::load_n<E, 4>(at + e0, false, x[u][0]);
                bq::load_n<E, 4>(at + e1, false, x[u][1]);
            }
        }
    };

    // this thread's pair, of every `at_once`-th token of a batch
    const int pair = tid % HALF_MAX, at_once = blockDim.x / HALF_MAX, mine = tid / HALF_MAX;
    const bool turns = pair < half && mine < at_once;
    int axis = 0;
    if (turns)
        axis = (pair >= a.x.sections[0] && a.x.axes > 1) +
               (pair >= a.x.sections[0] + a.x.sections[1] && a.x.axes > 2);
    float hi = 0.0f, lo = 0.0f;

    const long long stride = groups * a.batch;
    int n[MAX_BATCH];  // positions and a slot of the next batch
    long long slot = -1;
    auto look_up = [&](long long t0) {
        const long long left = a.x.tokens - t0;
#pragma unroll
        for (int k = 0; k < MAX_BATCH; ++k) {
            const int b = mine + k * at_once;
            n[k] = turns && b < a.batch && b < left ? a.x.positions[axis * a.x.position_stride + t0 + b] : 0;
        }
        slot = tid < a.batch && tid < left ? a.x.slots[t0 + tid] : -1;
    };
    const long long start = blockIdx.x / a.parts * (long long)a.batch;
#pragma unroll
    for (int b = 0; b < MAX_BATCH; ++b) fetch(b < a.batch ? start + b : a.x.tokens, b);
    look_up(start);
    if (turns) {
        const double t = a.x.freq[pair] * 0.15915494309189533576888;  // 1 / (2 pi)
        hi = (float)t;
        lo = (float)(t - (double)hi);
    }

    int buf = 0;
    for (long long t0 = start; t0 < a.x.tokens; t0 += stride, buf ^= 1) {
        const int batch = (int)(a.x.tokens - t0 < a.batch ? a.x.tokens - t0 : a.batch);
        // ---- slots and angles of the batch ----
        if (tid < batch) {
            long long row = -1;  // element offset of the token's slot, head 0
            if (slot >= 0 && slot < slots_all) {
                const long long page = slot <= 0x7fffffffLL ? (long long)a.page.div((uint32_t)slot)
                                                            : slot / a.c.page_size;
                row = page * (long long)a.page_s + (slot - page * a.c.page_size) * (long long)a.slot_s;
            } else if (slot >= slots_all && part == 0) {
                atomicOr(&g_status_append, BQ_DEVERR_SLOT);
            }
            row_s[buf][tid] = row;
        }
        if (turns) {
#pragma unroll
            for (int k = 0; k < MAX_BATCH; ++k) {
                const int b = mine + k * at_once;
                if (b >= batch) break;
                const float nf = (float)n[k];  // beyond 2^24 rounded: the rest is nr, exact
                const float nr = (float)((long long)n[k] - (long long)nf);
                const float p = __fmul_rn(nf, hi);
                const float e = __fmaf_rn(nf, hi, -p);
                float f = (p - rintf(p)) + (e - rintf(e));
                float rest = __fmul_rn(nf, lo);
                if (fabsf(nf) > 0x1p24f) {  // several turns, and nr: by product and remainder too
                    const float u = __fmul_rn(nr, hi);
                    const float left = __fmaf_rn(nf, lo, -rest) + __fmaf_rn(nr, hi, -u);
                    rest = ((rest - rintf(rest)) + (u - rintf(u))) + left;
                }
                f += rest - rintf(rest);
                float s, c;
                sincospif(2.0f * (f - rintf(f)), &s, &c);
                cs_s[buf][b][pair] = make_float2(c, s);
            }
        }
        __syncthreads();  // (the batch after the next rewrites this buffer, two barriers on)

        look_up(t0 + stride);
        // (unrolled, the quantizer's code outgrows the instruction cache: 8192 tokens 54 us against 50)
#pragma unroll (CT == BQ_Q8_0 ? 1 : MAX_BATCH)
        for (int b = 0; b < MAX_BATCH; ++b) {
            asm volatile("cp.async.wait_group %0;" ::"n"(MAX_BATCH - 1) : "memory");
            float y[UNROLL][2][4];
            if (b < batch) load((uint32_t)t0 + b, b, y);
            fetch(b < a.batch ? t0 + stride + b : a.x.tokens, b);
            if (b >= batch) continue;
            const uint32_t t = (uint32_t)t0 + b;
            const long long row = row_s[buf][b];
            float2 w[4];  // cosine and sine of this lane's four pairs
            if (in_rot) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float4 v = *reinterpret_cast<const float4 *>(&cs_s[buf][b][4 * i + 2 * k]);
                    w[2 * k] = make_float2(v.x, v.y), w[2 * k + 1] = make_float2(v.z, v.w);
                }
            }
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {
                float(&p)[4] = y[u][0], (&q)[4] = y[u][1];
                if (in_rot && type[u] < 2) {
                    if (apart) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float e = p[k], o = q[k];
                            p[k] = fmaf(o, -w[k].y, e * w[k].x);
                            q[k] = fmaf(e, w[k].y, o * w[k].x);
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            float(&z)[4] = y[u][k >> 1];
                            const float e = z[2 * (k & 1)], o = z[2 * (k & 1) + 1];
                            z[2 * (k & 1)] = fmaf(o, -w[k].y, e * w[k].x);
                            z[2 * (k & 1) + 1] = fmaf(e, w[k].y, o * w[k].x);
                        }
                    }
                }
                if (type[u] == 0 && there) {
                    T *dst = out[u] + (uint64_t)t * a.o_t;
                    bq::store_n<E, 4>(dst + e0, a.wide_out, p);
                    bq::store_n<E, 4>(dst + e1, a.wide_out, q);
                }
                const bool keep = there && row >= 0 && (type[u] == 1 || type[u] == 2);
                const long long at = row + (long long)((uint64_t)head_at[u] * a.head_s);
                void *plane = type[u] == 1 ? a.c.k : a.c.v;
                if constexpr (CT == BQ_Q8_0) {
                    if (!any_kept[u]) continue;  // only queries
                    int f0 = e0, f1 = e1;     // where the quarters lie
                    bool rows_of_8 = !apart;
                    if (half % 32 && !a.x.interleaved) {  // rotated halves cut blocks: put in order
                        float *mine = order_s + (warp * HPW + sub) * DMAX;
                        __syncwarp();
                        if (there) {
                            *reinterpret_cast<float4 *>(mine + e0) = make_float4(p[0], p[1], p[2], p[3]);
                            *reinterpret_cast<float4 *>(mine + e1) = make_float4(q[0], q[1], q[2], q[3]);
                        }
                        __syncwarp();
                        f0 = 8 * i, f1 = 8 * i + 4, rows_of_8 = true;
                        const float4 g0 = *reinterpret_cast<const float4 *>(mine + f0);
                        const float4 g1 = *reinterpret_cast<const float4 *>(mine + f1);
                        p[0] = g0.x, p[1] = g0.y, p[2] = g0.z, p[3] = g0.w;
                        q[0] = g1.x, q[1] = g1.y, q[2] = g1.z, q[3] = g1.w;
                    }
                    // the largest magnitude: a NaN counts only where there is nothing else
                    float m0 = NAN, m1 = NAN;
                    if (there) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) m0 = fmaxf(m0, fabsf(p[k])), m1 = fmaxf(m1, fabsf(q[k]));
                    }
                    if (rows_of_8) m0 = m1 = fmaxf(m0, m1);
#pragma unroll
                    for (int o = 1; o < 4; o <<= 1) {
                        m0 = fmaxf(m0, __shfl_xor_sync(~0u, m0, o));
                        m1 = fmaxf(m1, __shfl_xor_sync(~0u, m1, o));
                    }
                    const float n0 = __shfl_xor_sync(~0u, m0, 4), n1 = __shfl_xor_sync(~0u, m1, 4);
                    if (!rows_of_8) m0 = fmaxf(m0, n0), m1 = fmaxf(m1, n1);
                    if (keep) {
                        __half *scales = (__half *)(type[u] == 1 ? a.c.k_scale : a.c.v_scale);
                        auto quantize = [&](const float(&z)[4], float m, int f, bool writes_scale) {
                            const __half d = __float2half_rn(__fdiv_rn(m, 127.0f));
                            const float df = __half2float(d);
                            // a little below 1 / d (the quotient is good to 2 ulp), so that the
                            // guess is never too large
                            const float inv = __fdividef(1.0f - 0x1p-20f, df), half_d = 0.5f * df;
                            uint32_t c[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) c[k] = q8_code(z[k], df, half_d, inv);
                            const uint32_t word = __byte_perm(__byte_perm(c[0], c[1], 0x0040),
                                                              __byte_perm(c[2], c[3], 0x0040), 0x5410);
                            // (a scale of 0: the codes are 0)
                            *reinterpret_cast<uint32_t *>((uint8_t *)plane + at + f) = df != 0.0f ? word : 0u;
                            if (writes_scale) scales[(at + f) >> 5] = d;
                        };
                        quantize(p, m0, f0, (f0 & 31) == 0);
                        quantize(q, m1, f1, (f1 & 31) == 0);
                    }
                } else if (keep) {
                    using C = typename std::conditional<CT == BQ_F16, bq::F16, bq::BF16>::type;
                    bq::store_wide<C, 4>((typename C::T *)plane + at + e0, p);
                    bq::store_wide<C, 4>((typename C::T *)plane + at + e1, q);
                }
            }
        }
    }
}

// shared memory of a warp: its values on their way, and the heads put in order
constexpr int warp_smem(int element, bool order) {
    return MAX_BATCH * UNROLL * 2 * 32 * 4 * element + (order ? 32 * 8 * 4 : 0);
}

template <class E, int CT>
cudaError_t launch(const Args &a, int grid, void *stream) {
    auto *kern = a.c.head_dim <= 64    ? append_kernel<E, CT, 8>
                 : a.c.head_dim <= 128 ? append_kernel<E, CT, 16>
                                       : append_kernel<E, CT, 32>;
    if (a.smem > 24 * 1024) {  // (up to 9 KB of static shared memory beside it)
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   MAX_WARPS * warp_smem(4, true));
        if (e != cudaSuccess) return e;
    }
    return bq::launch_pdl(kern, dim3((unsigned)grid), a.warps * 32, (size_t)a.smem, stream, 1, a);
}
template <class E>
cudaError_t launch(const Args &a, int grid, void *stream) {
    return a.c.type == BQ_F16    ? launch<E, BQ_F16>(a, grid, stream)
           : a.c.type == BQ_BF16 ? launch<E, BQ_BF16>(a, grid, stream)
                                 : launch<E, BQ_Q8_0>(a, grid, stream);
}

bool stride_ok(int64_t s) { return s >= 0 && s <= 0x7fffffffLL; }

}  // namespace

namespace bq {
int device_sms() {
    static std::atomic<int> cache[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    int n = cache[dev].load();
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
        cache[dev].store(n);
    }
    return n;
}
}  // namespace bq

int bq_internal_status_append(unsigned int *flags, int clear) { return read_status_append(flags, clear); }

extern "C" bq_status bq_kv_append(const bq_kv_cache *cache, const bq_kv_append_args *x, void *stream) {
    if (!cache || !x) return BQ_ERR_NULL;
    bq_status s = bq::check_cache_shape(cache);
    if (s != BQ_OK) return s;
    const int es = bq::dtype_bytes(x->dtype);
    if (!es) return BQ_ERR_QTYPE;
    if (x->tokens < 0 || x->tokens > 0x7fffffffLL) return BQ_ERR_SHAPE;
    const int64_t strides[] = {x->k_token_stride, x->k_head_stride, x->v_token_stride, x->v_head_stride};
    for (int64_t v : strides)
        if (!stride_ok(v)) return BQ_ERR_SHAPE;
    if (x->q) {
        if (x->heads < 1 || x->heads > 4096) return BQ_ERR_SHAPE;
        const int64_t qs[] = {x->q_token_stride, x->q_head_stride, x->q_out_token_stride, x->q_out_head_stride};
        for (int64_t v : qs)
            if (!stride_ok(v)) return BQ_ERR_SHAPE;
    }
    if (x->freq) {
        if (x->rot < 16 || x->rot % 16 || x->rot > cache->head_dim || x->axes < 1 || x->axes > 3 ||
            !stride_ok(x->position_stride))
            return BQ_ERR_SHAPE;
        int64_t sum = 0;
        for (int i = 0; i < x->axes; ++i) {
            if (x->sections[i] < 0) return BQ_ERR_SHAPE;
            sum += x->sections[i];
        }
        if (sum != x->rot / 2) return BQ_ERR_SHAPE;
    }
    if (x->tokens == 0) return BQ_OK;
    s = bq::check_cache_pointers(cache);
    if (s != BQ_OK) return s;
    if (!x->k || !x->v || !x->slots || (x->q && !x->q_out) || (x->freq && !x->positions)) return BQ_ERR_NULL;
    const void *typed[] = {x->k, x->v, x->q, x->q ? x->q_out : nullptr};
    for (const void *p : typed)
        if (!bq::aligned_to(p, (uintptr_t)es)) return BQ_ERR_ALIGN;
    if (!bq::aligned_to(x->slots, 8) || (x->freq && (!bq::aligned_to(x->freq, 8) || !bq::aligned_to(x->positions, 4))))
        return BQ_ERR_ALIGN;
    const int sms = bq::device_sms();
    if (!sms) return BQ_ERR_CUDA;
    Args a;
    a.c = *cache;
    a.x = *x;
    a.page.set((uint32_t)cache->page_size);
    a.items = (x->q ? x->heads : 0) + 2 * cache->kv_heads;
    auto wide = [&](const void *p, int64_t t, int64_t h) {
        return bq::aligned_to(p, (uintptr_t)(4 * es)) && t % 4 == 0 && h % 4 == 0;
    };
    a.wide = wide(x->k, x->k_token_stride, x->k_head_stride) && wide(x->v, x->v_token_stride, x->v_head_stride) &&
             (!x->q || wide(x->q, x->q_token_stride, x->q_head_stride));
    a.wide_out = x->q && wide(x->q_out, x->q_out_token_stride, x->q_out_head_stride);
    a.q_t = (uint32_t)x->q_token_stride, a.q_h = (uint32_t)x->q_head_stride;
    a.k_t = (uint32_t)x->k_token_stride, a.k_h = (uint32_t)x->k_head_stride;
    a.v_t = (uint32_t)x->v_token_stride, a.v_h = (uint32_t)x->v_head_stride;
    a.o_t = (uint32_t)x->q_out_token_stride, a.o_h = (uint32_t)x->q_out_head_stride;
    a.page_s = (uint32_t)cache->page_stride, a.head_s = (uint32_t)cache->head_stride;
    a.slot_s = (uint32_t)cache->slot_stride;
    // A CTA has a warp for every 2 HPW heads of a token, and enough to turn a
    // token's pairs (a warp left over idles: 16000 tokens of 2 + 2 heads of 64 in
    // four warps 17 us, in one 10); more heads go to more CTAs, each with the angles
    // once more.
    const int gl = cache->head_dim <= 64 ? 8 : cache->head_dim <= 128 ? 16 : 32;
    const int of_warp = UNROLL * (32 / gl);
    const int warps = (a.items + of_warp - 1) / of_warp;
    a.parts = (warps + MAX_WARPS - 1) / MAX_WARPS;
    a.warps = (warps + a.parts - 1) / a.parts;
    const int least = 4 * gl / 32;
    if (a.warps < least) a.warps = least;
    // as many CTAs as are resident together (24 warps of 80 registers per SM, 227 KB
    // of shared memory with the angles and 1 KB of each CTA's own), at MAX_BATCH
    // tokens at a time if there are that many
    const bool order = cache->type == BQ_Q8_0 && x->freq && x->rot / 2 % 32 && !x->interleaved;
    a.smem = a.warps * warp_smem(es, order);
    const int by_smem = 228 * 1024 / (a.smem + 2 * MAX_BATCH * 4 * gl * 8 + 1024 + 256);
    const long long fit = (long long)sms * (24 / a.warps < by_smem ? 24 / a.warps : by_smem);
    const long long each = (x->tokens * a.parts + fit - 1) / fit;
    a.batch = each < 1 ? 1 : each > MAX_BATCH ? MAX_BATCH : (int)each;
    const long long groups = (x->tokens + a.batch - 1) / a.batch;
    const long long most = (fit + a.parts - 1) / a.parts;
    const int grid = (int)(groups < most ? groups : most) * a.parts;
    return bq::from_cuda_error(x->dtype == BQ_F32   ? launch<bq::F32>(a, grid, stream)
                               : x->dtype == BQ_F16 ? launch<bq::F16>(a, grid, stream)
                                                    : launch<bq::BF16>(a, grid, stream));
}
