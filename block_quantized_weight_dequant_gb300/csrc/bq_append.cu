// bq_append.cu -- keys and values of new tokens into the paged cache, with
// rotary positions of one to three axes (bq_kv_append in include/bqgemv.h).
//
// Angles: the turn of pair p at position n is n * freq / (2 pi).  freq/(2 pi)
// is split once per warp into hi + lo (two fp32 words, 48 bits); per token
// n * hi is formed exactly as product and remainder (one FMUL, one FFMA), each
// reduced by its nearest whole number, so the fraction of a turn is right to
// about 2^-24 of a turn plus n * freq * 2^-48, at positions up to 2^31.  fp64
// runs once per warp and pair only (its rate is far below fp32's).
//
// One warp takes a head of a token: lane l holds elements 4l .. 4l+3 (and
// 128 + 4l .. for heads over 128), one 16-byte load of fp32; the partner of a
// (p, p + rot/2) pair comes by shuffle, a Q8_0 block is 8 lanes.  A warp stays
// with one residue of the heads over the tokens that it takes, so its angles
// serve all its heads of a token; with few tokens there is a warp for every
// head.  Bound by HBM for a prompt, by latency for one token.
#include <atomic>
#include <type_traits>

#include "bq_cache.cuh"

namespace {

BQ_STATUS_WORD(append)

constexpr int THREADS = 128;
constexpr int UNROLL = 4;  // heads in flight per warp

struct Args {
    bq_kv_cache c;
    bq_kv_append_args x;
    bq::FastDiv page;
    int items;  // heads of a token: q, k and v
    int parts;  // warps that share a token's heads
    int wide_k, wide_v, wide_q, wide_o;  // 4-element accesses allowed
};

// pair and partner of element e < rot
struct Place {
    int pair, partner;
    bool second;  // the pair's second element
};
__device__ __forceinline__ Place place_of(int e, int rot, int interleaved) {
    const int half = rot >> 1;
    Place p;
    if (interleaved) {
        p.pair = e >> 1;
        p.partner = e ^ 1;
        p.second = e & 1;
    } else {
        p.second = e >= half;
        p.pair = p.second ? e - half : e;
        p.partner = p.second ? e - half : e + half;
    }
    return p;
}

template <class E, int CT, int ITS>
__global__ void __launch_bounds__(THREADS) append_kernel(const __grid_constant__ Args a) {
    using T = typename E::T;
    const int lane = threadIdx.x & 31;
    const int warps = gridDim.x * (THREADS / 32);
    const int wid = blockIdx.x * (THREADS / 32) + (threadIdx.x >> 5);
    const int part = wid % a.parts;
    const int step = warps / a.parts;
    const long long first = wid / a.parts;
    bq::pdl_wait();
    if (first >= step) return;

    const int D = a.c.head_dim, rot = a.x.freq ? a.x.rot : 0, half = rot >> 1;
    float hi[ITS][4], lo[ITS][4];
    int axis[ITS][4];
#pragma unroll
    for (int it = 0; it < ITS; ++it)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = 128 * it + 4 * lane + i;
            hi[it][i] = lo[it][i] = 0.0f;
            axis[it][i] = 0;
            if (e < rot) {
                const int p = place_of(e, rot, a.x.interleaved).pair;
                const double t = a.x.freq[p] * 0.15915494309189533576888;  // 1 / (2 pi)
                hi[it][i] = (float)t;
                lo[it][i] = (float)(t - (double)hi[it][i]);
                axis[it][i] = (p >= a.x.sections[0] && a.x.axes > 1) +
                              (p >= a.x.sections[0] + a.x.sections[1] && a.x.axes > 2);
            }
        }

    const int heads = a.x.q ? a.x.heads : 0, kv = a.c.kv_heads;
    const long long slots_all = a.c.pages * a.c.page_size;
    for (long long t = first; t < a.x.tokens; t += step) {
        const long long slot = a.x.slots[t];
        long long row = -1;  // element offset of the token's slot, head 0
        if (slot >= 0 && slot < slots_all) {
            const long long page = slot <= 0x7fffffffLL ? (long long)a.page.div((uint32_t)slot)
                                                        : slot / a.c.page_size;
            row = page * a.c.page_stride + (slot - page * a.c.page_size) * a.c.slot_stride;
        } else if (slot >= slots_all && lane == 0) {
            atomicOr(&g_status_append, BQ_DEVERR_SLOT);
        }
        float cs[ITS][4], sn[ITS][4];
        if (rot) {
            float pf[3], pr[3];
#pragma unroll
            for (int x = 0; x < 3; ++x) {
                const int n = x < a.x.axes ? a.x.positions[x * a.x.position_stride + t] : 0;
                pf[x] = (float)n;  // beyond 2^24 rounded: the rest is pr, exact
                pr[x] = (float)((long long)n - (long long)pf[x]);
            }
#pragma unroll
            for (int it = 0; it < ITS; ++it)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int ax = axis[it][i];
                    const float n = ax == 0 ? pf[0] : ax == 1 ? pf[1] : pf[2];
                    const float r = ax == 0 ? pr[0] : ax == 1 ? pr[1] : pr[2];
                    const float p = __fmul_rn(n, hi[it][i]);
                    const float e = __fmaf_rn(n, hi[it][i], -p);
                    float f = (p - rintf(p)) + (e - rintf(e));
                    const float rest = __fmaf_rn(n, lo[it][i], r * hi[it][i]);
                    f += rest - rintf(rest);
                    sincospif(2.0f * (f - rintf(f)), &sn[it][i], &cs[it][i]);
                }
        }
        for (int i0 = part; i0 < a.items; i0 += UNROLL * a.parts) {
            float x[UNROLL][ITS][4];
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {
                const int item = i0 + u * a.parts;
                if (item >= a.items || (item >= heads && row < 0)) continue;
                const T *src;
                int wide;
                if (item < heads) {
                    src = (const T *)a.x.q + t * a.x.q_token_stride + item * a.x.q_head_stride;
                    wide = a.wide_q;
                } else if (item < heads + kv) {
                    src = (const T *)a.x.k + t * a.x.k_token_stride + (item - heads) * a.x.k_head_stride;
                    wide = a.wide_k;
                } else {
                    src = (const T *)a.x.v + t * a.x.v_token_stride + (item - heads - kv) * a.x.v_head_stride;
                    wide = a.wide_v;
                }
#pragma unroll
                for (int it = 0; it < ITS; ++it) {
                    const int e = 128 * it + 4 * lane;
                    if (e < D) bq::load_n<E, 4>(src + e, wide, x[u][it]);
                }
            }
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {
                const int item = i0 + u * a.parts;
                if (item >= a.items || (item >= heads && row < 0)) continue;
                float y[ITS][4];
                if (rot && item < heads + kv) {
#pragma unroll
                    for (int it = 0; it < ITS; ++it) {
                        const int e = 128 * it + 4 * lane;
                        float z[4];
                        if (a.x.interleaved) {
                            z[0] = x[u][it][1], z[1] = x[u][it][0], z[2] = x[u][it][3], z[3] = x[u][it][2];
                        } else {
                            // rot / 2 is a multiple of 4: the four partners are one lane's
                            const int pe = e >= half ? e - half : e + half;
                            const int from = (pe >> 2) & 31;
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                z[i] = __shfl_sync(~0u, x[u][0][i], from);
                                if constexpr (ITS == 2) {
                                    const float z1 = __shfl_sync(~0u, x[u][1][i], from);
                                    if (pe >= 128) z[i] = z1;
                                }
                            }
                        }
                        const bool turn = e < rot;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const bool second = a.x.interleaved ? (i & 1) : e >= half;
                            const float s = second ? sn[it][i] : -sn[it][i];
                            y[it][i] = turn ? fmaf(z[i], s, x[u][it][i] * cs[it][i]) : x[u][it][i];
                        }
                    }
                } else {
#pragma unroll
                    for (int it = 0; it < ITS; ++it)
#pragma unroll
                        for (int i = 0; i < 4; ++i) y[it][i] = x[u][it][i];
                }
                if (item < heads) {
                    T *dst = (T *)a.x.q_out + t * a.x.q_out_token_stride + item * a.x.q_out_head_stride;
#pragma unroll
                    for (int it = 0; it < ITS; ++it) {
                        const int e = 128 * it + 4 * lane;
                        if (e < D) bq::store_n<E, 4>(dst + e, a.wide_o, y[it]);
                    }
                    continue;
                }
                const bool is_k = item < heads + kv;
                const long long at = row + (item - heads - (is_k ? 0 : kv)) * a.c.head_stride;
                void *plane = is_k ? a.c.k : a.c.v;
#pragma unroll
                for (int it = 0; it < ITS; ++it) {
                    const int e = 128 * it + 4 * lane;
                    if constexpr (CT == BQ_Q8_0) {
                        float m = 0.0f;
#pragma unroll
                        for (int i = 0; i < 4; ++i) m = e < D ? fmaxf(m, fabsf(y[it][i])) : 0.0f;
#pragma unroll
                        for (int o = 1; o < 8; o <<= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
                        const __half d = __float2half_rn(__fdiv_rn(m, 127.0f));
                        const float df = __half2float(d);
                        uint32_t word = 0;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            int q = 0;
                            if (df != 0.0f)
                                q = (int)fminf(fmaxf(roundf(__fdiv_rn(y[it][i], df)), -127.0f), 127.0f);
                            word |= (uint32_t)(q & 0xff) << (8 * i);
                        }
                        if (e < D) {
                            *reinterpret_cast<uint32_t *>((uint8_t *)plane + at + e) = word;
                            if ((lane & 7) == 0)
                                ((__half *)(is_k ? a.c.k_scale : a.c.v_scale))[(at + e) >> 5] = d;
                        }
                    } else {
                        using C = typename std::conditional<CT == BQ_F16, bq::F16, bq::BF16>::type;
                        if (e < D) bq::store_n<C, 4>((typename C::T *)plane + at + e, true, y[it]);
                    }
                }
            }
        }
    }
}

template <class E, int CT>
cudaError_t launch(const Args &a, int grid, void *stream) {
    return a.c.head_dim <= 128
               ? bq::launch_pdl(append_kernel<E, CT, 1>, dim3((unsigned)grid), THREADS, 0, stream, 1, a)
               : bq::launch_pdl(append_kernel<E, CT, 2>, dim3((unsigned)grid), THREADS, 0, stream, 1, a);
}
template <class E>
cudaError_t launch(const Args &a, int grid, void *stream) {
    return a.c.type == BQ_F16    ? launch<E, BQ_F16>(a, grid, stream)
           : a.c.type == BQ_BF16 ? launch<E, BQ_BF16>(a, grid, stream)
                                 : launch<E, BQ_Q8_0>(a, grid, stream);
}

bool stride_ok(int64_t s) { return s >= 0 && s <= (1LL << 40); }

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
        if (x->rot < 8 || x->rot % 8 || x->rot > cache->head_dim || x->axes < 1 || x->axes > 3 ||
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
    a.wide_k = wide(x->k, x->k_token_stride, x->k_head_stride);
    a.wide_v = wide(x->v, x->v_token_stride, x->v_head_stride);
    a.wide_q = x->q && wide(x->q, x->q_token_stride, x->q_head_stride);
    a.wide_o = x->q && wide(x->q_out, x->q_out_token_stride, x->q_out_head_stride);
    // a warp for every head while that many warps fit the GPU, then fewer per token
    const long long fit = (long long)sms * 32;
    long long parts = (fit + x->tokens - 1) / x->tokens;
    a.parts = (int)(parts < a.items ? parts : a.items);
    long long warps = x->tokens * a.parts;
    const long long most = fit > a.parts ? fit : a.parts;
    if (warps > most) warps = most / a.parts * a.parts;
    const int grid = (int)((warps + THREADS / 32 - 1) / (THREADS / 32));
    return bq::from_cuda_error(x->dtype == BQ_F32   ? launch<bq::F32>(a, grid, stream)
                               : x->dtype == BQ_F16 ? launch<bq::F16>(a, grid, stream)
                                                    : launch<bq::BF16>(a, grid, stream));
}
