// bq_norm.cu -- the norms after one block and before the next with the block's
// gate and the residual scales, in one pass over the row (bq_sandwich_norm in
// include/bqgemv.h).
//
// A row is read once and kept in registers over both sums of squares: thread t
// of N holds the 8-element vectors t, t + N, ...; N and the vectors per thread
// follow from the width alone, and so does the order of every sum (each
// thread's vectors, a butterfly over the warp, the warps in order).  A row's
// bits are the same whichever rows are computed beside it.  Bound by HBM for
// many rows, by two block-wide sums and the launch for one.  Measured: 8192 rows
// of 5120, bf16 beside an fp32 residual: 86 us, 5.8 TB/s; one row of 1024: 2.0 us.
//
// Three instances of the one kernel differ in how a row reaches the registers:
//  ONCE   rows of whole aligned vectors, a CTA per row: direct loads.
//  AHEAD  the same with more rows than CTAs: a thread copies its own vectors of
//         the CTA's next row into shared memory (cp.async) before it works on
//         the present one, so loads are in flight across the two sums; a thread
//         reads only what it copied, so no barrier goes with it.  The gains (and
//         a gate per channel) are copied the same way once, where two CTAs per SM
//         still fit: read again for every row they cost an L2 latency after
//         each sum.
//  RAGGED any width and alignment, a CTA per row: element by element with a warp's
//         lanes side by side, put in the threads' order (and back) through 1 KB
//         of shared memory per warp.
#include "bq_cache.cuh"

#include <cmath>

namespace {

constexpr int MAX_WIDTH = 16384;

struct Args {
    bq_sandwich_args x;
    int wide;       // whole 16-byte vectors throughout
    int wide_gain;  // the gains are aligned to them
    int gains_s;    // AHEAD: gains and gate kept in shared memory
};

__device__ __forceinline__ float block_sum(float v, float *sm) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    if (blockDim.x == 32) return v;
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.0f;
    for (int w = 0; w < (int)(blockDim.x >> 5); ++w) s += sm[w];
    return s;
}

// 8 elements to shared memory, asynchronously
template <class E>
__device__ __forceinline__ void copy8(typename E::T *dst, const typename E::T *src) {
    const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(src) : "memory");
    if constexpr (sizeof(typename E::T) == 4)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + 16), "l"(src + 4) : "memory");
}

// A warp's 256 elements from lanes side by side (element 32 i + lane in x[i]) to
// eight in a row per lane, and back
__device__ __forceinline__ void to_rows(float *warp_s, int lane, float (&x)[8]) {
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i) warp_s[32 * i + lane] = x[i];
    __syncwarp();
    bq::load_wide<bq::F32, 8>(warp_s + 8 * lane, x);
}
__device__ __forceinline__ void to_lanes(float *warp_s, int lane, float (&x)[8]) {
    __syncwarp();
    bq::store_wide<bq::F32, 8>(warp_s + 8 * lane, x);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = warp_s[32 * i + lane];
}

constexpr int MAX_THREADS = 512;
enum { ONCE, AHEAD, RAGGED };

template <class EY, class EH, int VPT, int MODE>
__global__ void __launch_bounds__(MAX_THREADS, VPT <= 2 ? 2 : 1) sandwich_kernel(const __grid_constant__ Args a) {
    using TY = typename EY::T;
    using TH = typename EH::T;
    extern __shared__ __align__(16) uint8_t rows_s[];
    __shared__ float sm[2][32];
    const int width = (int)a.x.width, n = blockDim.x, tid = threadIdx.x;
    const float inv_width = 1.0f / (float)width;
    // AHEAD: two rows, h then y; RAGGED: 256 floats per warp
    const int row_elems = n * VPT * 8;
    TH *h_s = reinterpret_cast<TH *>(rows_s);
    TY *y_s = reinterpret_cast<TY *>(rows_s + 2 * row_elems * sizeof(TH));
    const int lane = tid & 31;
    float *warp_s = reinterpret_cast<float *>(rows_s) + 256 * (tid >> 5);
    // first element of this warp's v-th 256, less its lane
    auto side_by_side = [&](int v) { return 8 * ((tid & ~31) + v * n) + lane; };
    // this thread's vectors of a row
    auto fetch = [&](long long row, int k) {
        if (row < a.x.rows) {
            const TY *y = (const TY *)a.x.y + row * a.x.y_stride;
            const TH *h = (const TH *)a.x.h + row * a.x.h_stride;
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                const int at = 8 * (tid + v * n);
                if (at < width) {
                    copy8<EY>(y_s + k * row_elems + at, y + at);
                    copy8<EH>(h_s + k * row_elems + at, h + at);
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    const bool gate_s = a.gains_s && a.x.gate && a.x.gate_stride == 0;
    float *post_s = reinterpret_cast<float *>(rows_s + 2 * row_elems * (sizeof(TH) + sizeof(TY)));
    float *pre_s = post_s + row_elems;
    TY *gates_s = reinterpret_cast<TY *>(pre_s + row_elems);
    // factors of this thread's elements, read by 16 bytes where the row is whole vectors
    auto factor = [&](auto tag, const auto *p, int at, float(&g)[8]) {
        using E = decltype(tag);
        if (MODE != RAGGED || (at + 8 <= width && a.wide_gain)) {
            bq::load_wide<E, 8>(p + at, g);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) g[i] = at + i < width ? E::up(p[at + i]) : 0.0f;
        }
    };
    bq::pdl_wait();
    if constexpr (MODE == AHEAD) {
        if (a.gains_s) {
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                const int at = 8 * (tid + v * n);
                if (at < width) {
                    if (a.x.post) copy8<bq::F32>(post_s + at, a.x.post + at);
                    if (a.x.pre) copy8<bq::F32>(pre_s + at, a.x.pre + at);
                    if (gate_s) copy8<EY>(gates_s + at, (const TY *)a.x.gate + at);
                }
            }
        }
        fetch(blockIdx.x, 0);
    }
    int k = 0;
    for (long long row = blockIdx.x; row < a.x.rows; row += gridDim.x, k ^= 1) {
        const TY *y = (const TY *)a.x.y + row * a.x.y_stride;
        const TH *h = (const TH *)a.x.h + row * a.x.h_stride;
        float b[VPT][8], r[VPT][8];
        if constexpr (MODE == AHEAD) {
            fetch(row + gridDim.x, k ^ 1);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
        }
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int at = 8 * (tid + v * n);
            if constexpr (MODE == RAGGED) {
                const int e = side_by_side(v);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    b[v][i] = e + 32 * i < width ? EY::up(y[e + 32 * i]) : 0.0f;
                    r[v][i] = e + 32 * i < width ? EH::up(h[e + 32 * i]) : 0.0f;
                }
            } else if (at < width) {
                bq::load_wide<EY, 8>(MODE == AHEAD ? y_s + k * row_elems + at : y + at, b[v]);
                bq::load_wide<EH, 8>(MODE == AHEAD ? h_s + k * row_elems + at : h + at, r[v]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) b[v][i] = r[v][i] = 0.0f;
            }
        }
        if constexpr (MODE == RAGGED) {
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                to_rows(warp_s, lane, b[v]);
                to_rows(warp_s, lane, r[v]);
            }
        }
        if (a.x.post) {
            float s = 0.0f;
#pragma unroll
            for (int v = 0; v < VPT; ++v)
#pragma unroll
                for (int i = 0; i < 8; ++i) s = fmaf(b[v][i], b[v][i], s);
            const float scale = rsqrtf(fmaf(block_sum(s, sm[0]), inv_width, a.x.eps));
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                const int at = 8 * (tid + v * n);
                if (at < width) {
                    float g[8];
                    factor(bq::F32{}, MODE == AHEAD && a.gains_s ? post_s : a.x.post, at, g);
#pragma unroll
                    for (int i = 0; i < 8; ++i) b[v][i] *= scale * g[i];
                }
            }
        }
        if (a.x.gate) {
            const TY *gate = (const TY *)a.x.gate + row * a.x.gate_stride;
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                const int at = 8 * (tid + v * n);
                if (MODE == RAGGED || at < width) {
                    float g[8];
                    if constexpr (MODE == RAGGED) {
                        const int e = side_by_side(v);
#pragma unroll
                        for (int i = 0; i < 8; ++i) g[i] = e + 32 * i < width ? EY::up(gate[e + 32 * i]) : 0.0f;
                        to_rows(warp_s, lane, g);
                    } else {
                        factor(EY{}, MODE == AHEAD && gate_s ? gates_s : gate, at, g);
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) b[v][i] *= g[i];
                }
            }
        }
        TH *ho = (TH *)a.x.h_out + row * a.x.h_out_stride;
        float s = 0.0f;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int at = 8 * (tid + v * n);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                r[v][i] = fmaf(a.x.alpha, r[v][i], a.x.beta * b[v][i]);
                s = fmaf(r[v][i], r[v][i], s);
            }
            if constexpr (MODE == RAGGED) {
                float o[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = r[v][i];
                to_lanes(warp_s, lane, o);
                const int e = side_by_side(v);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (e + 32 * i < width) ho[e + 32 * i] = EH::down(o[i]);
            } else if (at < width) {
                bq::store_wide<EH, 8>(ho + at, r[v]);
            }
        }
        TY *x = (TY *)a.x.x + (a.x.x ? row * a.x.x_stride : 0);
        if (a.x.x) {
            const float scale = rsqrtf(fmaf(block_sum(s, sm[1]), inv_width, a.x.eps));
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                const int at = 8 * (tid + v * n);
                if (MODE == RAGGED || at < width) {
                    float g[8];
                    factor(bq::F32{}, MODE == AHEAD && a.gains_s ? pre_s : a.x.pre, at, g);
#pragma unroll
                    for (int i = 0; i < 8; ++i) g[i] *= r[v][i] * scale;
                    if constexpr (MODE == RAGGED) {
                        to_lanes(warp_s, lane, g);
                        const int e = side_by_side(v);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (e + 32 * i < width) x[e + 32 * i] = EY::down(g[i]);
                    } else {
                        bq::store_wide<EY, 8>(x + at, g);
                    }
                }
            }
        }
        if (!(a.x.post && a.x.x)) {
            // the next row's sums reuse sm: with both, sm[0] is rewritten only after every
            // warp has passed the barrier inside block_sum on sm[1], and the other way round
            __syncthreads();
        }
    }
}

template <class EY, class EH, int VPT>
cudaError_t launch_vpt(const Args &a, int threads, int sms, void *stream) {
    const int elems = threads * VPT * 8;
    const size_t ahead = (size_t)2 * elems * (sizeof(typename EY::T) + sizeof(typename EH::T));
    if (!a.wide) {
        return bq::launch_pdl(sandwich_kernel<EY, EH, VPT, RAGGED>, dim3((unsigned)a.x.rows), threads,
                              (size_t)threads * 32, stream, 1, a);
    }
    // CTAs per SM: two rows of shared memory each and, where two CTAs fit with
    // them, the gains; else about 48 KB are left to L1 for those
    constexpr int MOST_THREADS = VPT <= 2 ? 1024 : 512;
    const size_t gains = (size_t)elems * (8 + sizeof(typename EY::T));
    const bool gains_s = 2 * (ahead + gains + 1280) <= 228 * 1024;
    const size_t smem = ahead + (gains_s ? gains : 0);
    int fit = (int)((gains_s ? 228 * 1024 : 176 * 1024) / (smem + 1280));
    if (fit > MOST_THREADS / threads) fit = MOST_THREADS / threads;
    if (fit < 1) fit = 1;
    const long long most = (long long)sms * fit;
    // Rows ahead pay where the gains are kept or two rows leave L1 room for them
    // (72 KB a CTA), and where 32 elements a thread leave one CTA per SM; else the
    // hardware's next CTA hides as much (fp32 rows of 8192: 126 us against 158).
    constexpr size_t MOST_AHEAD = 200 * 1024;
    const bool pays = gains_s || VPT == 4 || ahead <= 72 * 1024;
    if (a.x.rows <= most || smem > MOST_AHEAD || !pays)
        return bq::launch_pdl(sandwich_kernel<EY, EH, VPT, ONCE>, dim3((unsigned)a.x.rows), threads, 0, stream, 1, a);
    auto *kern = sandwich_kernel<EY, EH, VPT, AHEAD>;
    if (smem > 48 * 1024) {
        const cudaError_t e =
            cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)MOST_AHEAD);
        if (e != cudaSuccess) return e;
    }
    Args with = a;
    with.gains_s = gains_s;
    return bq::launch_pdl(kern, dim3((unsigned)most), threads, smem, stream, 1, with);
}

template <class EY, class EH>
cudaError_t launch(const Args &a, int sms, void *stream) {
    const int vecs = (int)((a.x.width + 7) / 8);
    // vectors per thread: one up to 2048 values, two up to 8192, four beyond
    const int vpt = vecs <= 256 ? 1 : vecs <= 1024 ? 2 : 4;
    const int threads = ((vecs + vpt - 1) / vpt + 31) / 32 * 32;
    return vpt == 1   ? launch_vpt<EY, EH, 1>(a, threads, sms, stream)
           : vpt == 2 ? launch_vpt<EY, EH, 2>(a, threads, sms, stream)
                      : launch_vpt<EY, EH, 4>(a, threads, sms, stream);
}

}  // namespace

extern "C" bq_status bq_sandwich_norm(const bq_sandwich_args *x, void *stream) {
    if (!x) return BQ_ERR_NULL;
    const int ey = bq::dtype_bytes(x->dtype), eh = bq::dtype_bytes(x->h_dtype);
    if (!ey || !eh || (x->h_dtype != BQ_F32 && x->h_dtype != x->dtype)) return BQ_ERR_QTYPE;
    if (x->rows < 0 || x->rows > 0x7fffffffLL || x->width < 1 || x->width > MAX_WIDTH) return BQ_ERR_SHAPE;
    const int64_t strides[] = {x->y_stride, x->h_stride, x->gate_stride, x->h_out_stride, x->x_stride};
    for (int64_t s : strides)
        if (s < 0 || s > 0x7fffffffLL) return BQ_ERR_SHAPE;
    if (!(std::isfinite(x->eps) && x->eps >= 0.0f) || !std::isfinite(x->alpha) || !std::isfinite(x->beta))
        return BQ_ERR_SHAPE;
    if (x->rows == 0) return BQ_OK;
    if (!x->y || !x->h || !x->h_out || (x->x && !x->pre)) return BQ_ERR_NULL;
    const void *typed[] = {x->y, x->gate, x->x};
    for (const void *p : typed)
        if (!bq::aligned_to(p, (uintptr_t)ey)) return BQ_ERR_ALIGN;
    if (!bq::aligned_to(x->h, (uintptr_t)eh) || !bq::aligned_to(x->h_out, (uintptr_t)eh) ||
        !bq::aligned_to(x->post, 4) || !bq::aligned_to(x->pre, 4))
        return BQ_ERR_ALIGN;
    if (x->x == x->h_out) return BQ_ERR_SHAPE;  // one would be written over the other
    const int sms = bq::device_sms();
    if (!sms) return BQ_ERR_CUDA;
    Args a;
    a.x = *x;
    // rows of 8-element vectors: the base pointers and, with several rows, the strides
    auto row_ok = [&](const void *p, int64_t stride) {
        return bq::aligned_to(p, 16) && (x->rows == 1 || stride % 8 == 0);
    };
    a.gains_s = 0;
    a.wide_gain = bq::aligned_to(x->post, 16) && bq::aligned_to(x->pre, 16);
    a.wide = x->width % 8 == 0 && row_ok(x->y, x->y_stride) && row_ok(x->gate, x->gate_stride) &&
             row_ok(x->x, x->x_stride) && row_ok(x->h, x->h_stride) && row_ok(x->h_out, x->h_out_stride) && a.wide_gain;
    cudaError_t e;
    if (x->dtype == BQ_F32)
        e = launch<bq::F32, bq::F32>(a, sms, stream);
    else if (x->dtype == BQ_F16)
        e = x->h_dtype == BQ_F32 ? launch<bq::F16, bq::F32>(a, sms, stream)
                                 : launch<bq::F16, bq::F16>(a, sms, stream);
    else
        e = x->h_dtype == BQ_F32 ? launch<bq::BF16, bq::F32>(a, sms, stream)
                                 : launch<bq::BF16, bq::BF16>(a, sms, stream);
    return bq::from_cuda_error(e);
}
