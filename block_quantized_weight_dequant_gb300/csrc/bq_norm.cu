// bq_norm.cu -- the norms after one block and before the next with the block's
// gate and the residual scales, in one pass over the row (bq_sandwich_norm in
// include/bqgemv.h).
//
// A row is read once and kept in registers over both sums of squares: thread t
// of N holds the 4-element vectors t, t + N, ...; N and the vectors per thread
// follow from the width alone, and so does the order of every sum (each
// thread's vectors, a butterfly over the warp, the warps in order).  A row's
// bits are the same whichever rows are computed beside it.  Bound by HBM for
// many rows, by two block-wide sums and the launch for one.
#include "bq_cache.cuh"

#include <cmath>

namespace {

constexpr int MAX_WIDTH = 16384;

struct Args {
    bq_sandwich_args x;
    int wide;  // 4-element accesses of the rows allowed
    int wide_gain;
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

template <class E, int N>
__device__ __forceinline__ void load_part(const typename E::T *p, int at, int width, bool wide, float (&out)[N]) {
    if (at + N <= width) {
        bq::load_n<E, N>(p + at, wide, out);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) out[i] = at + i < width ? E::up(p[at + i]) : 0.0f;
    }
}
template <class E, int N>
__device__ __forceinline__ void store_part(typename E::T *p, int at, int width, bool wide, const float (&in)[N]) {
    if (at + N <= width) {
        bq::store_n<E, N>(p + at, wide, in);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (at + i < width) p[at + i] = E::down(in[i]);
    }
}

template <class EY, class EH, int VPT>
__global__ void sandwich_kernel(const __grid_constant__ Args a) {
    using TY = typename EY::T;
    using TH = typename EH::T;
    __shared__ float sm[2][32];
    const int width = (int)a.x.width, n = blockDim.x;
    const bool wide = a.wide, wg = a.wide_gain;
    bq::pdl_wait();
    for (long long row = blockIdx.x; row < a.x.rows; row += gridDim.x) {
        const TY *y = (const TY *)a.x.y + row * a.x.y_stride;
        const TH *h = (const TH *)a.x.h + row * a.x.h_stride;
        float b[VPT][4], r[VPT][4];
#pragma unroll
        for (int v = 0; v < VPT; ++v) load_part<EY, 4>(y, 4 * (threadIdx.x + v * n), width, wide, b[v]);
#pragma unroll
        for (int v = 0; v < VPT; ++v) load_part<EH, 4>(h, 4 * (threadIdx.x + v * n), width, wide, r[v]);
        if (a.x.post) {
            float s = 0.0f;
#pragma unroll
            for (int v = 0; v < VPT; ++v)
#pragma unroll
                for (int i = 0; i < 4; ++i) s = fmaf(b[v][i], b[v][i], s);
            const float scale = rsqrtf(block_sum(s, sm[0]) / (float)width + a.x.eps);
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                float g[4];
                load_part<bq::F32, 4>(a.x.post, 4 * (threadIdx.x + v * n), width, wg, g);
#pragma unroll
                for (int i = 0; i < 4; ++i) b[v][i] = b[v][i] * scale * g[i];
            }
        }
        if (a.x.gate) {
            const TY *gate = (const TY *)a.x.gate + row * a.x.gate_stride;
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                float g[4];
                load_part<EY, 4>(gate, 4 * (threadIdx.x + v * n), width, wide, g);
#pragma unroll
                for (int i = 0; i < 4; ++i) b[v][i] *= g[i];
            }
        }
        TH *ho = (TH *)a.x.h_out + row * a.x.h_out_stride;
        float s = 0.0f;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                r[v][i] = fmaf(a.x.alpha, r[v][i], a.x.beta * b[v][i]);
                s = fmaf(r[v][i], r[v][i], s);
            }
            store_part<EH, 4>(ho, 4 * (threadIdx.x + v * n), width, wide, r[v]);
        }
        if (a.x.x) {
            const float scale = rsqrtf(block_sum(s, sm[1]) / (float)width + a.x.eps);
            TY *x = (TY *)a.x.x + row * a.x.x_stride;
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                float g[4];
                load_part<bq::F32, 4>(a.x.pre, 4 * (threadIdx.x + v * n), width, wg, g);
#pragma unroll
                for (int i = 0; i < 4; ++i) g[i] = r[v][i] * scale * g[i];
                store_part<EY, 4>(x, 4 * (threadIdx.x + v * n), width, wide, g);
            }
        }
        // the next row's sums reuse sm: sm[0] is rewritten only after every warp
        // has passed the barrier inside block_sum on sm[1], and the other way round
        if (!(a.x.post && a.x.x)) __syncthreads();
    }
}

template <class EY, class EH>
cudaError_t launch(const Args &a, int sms, void *stream) {
    const int vecs = (int)((a.x.width + 3) / 4);
    // vectors per thread: one up to 2048 values, two up to 4096, four beyond
    const int vpt = vecs <= 512 ? 1 : vecs <= 1024 ? 2 : 4;
    const int threads = ((vecs + vpt - 1) / vpt + 31) / 32 * 32;
    long long grid = a.x.rows;
    const long long most = (long long)sms * (2048 / threads);
    if (grid > most) grid = most;
    auto kern = vpt == 1   ? sandwich_kernel<EY, EH, 1>
                : vpt == 2 ? sandwich_kernel<EY, EH, 2>
                           : sandwich_kernel<EY, EH, 4>;
    return bq::launch_pdl(kern, dim3((unsigned)grid), threads, 0, stream, 1, a);
}

}  // namespace

extern "C" bq_status bq_sandwich_norm(const bq_sandwich_args *x, void *stream) {
    if (!x) return BQ_ERR_NULL;
    const int ey = bq::dtype_bytes(x->dtype), eh = bq::dtype_bytes(x->h_dtype);
    if (!ey || !eh || (x->h_dtype != BQ_F32 && x->h_dtype != x->dtype)) return BQ_ERR_QTYPE;
    if (x->rows < 0 || x->rows > 0x7fffffffLL || x->width < 1 || x->width > MAX_WIDTH) return BQ_ERR_SHAPE;
    const int64_t strides[] = {x->y_stride, x->h_stride, x->gate_stride, x->h_out_stride, x->x_stride};
    for (int64_t s : strides)
        if (s < 0 || s > (1LL << 40)) return BQ_ERR_SHAPE;
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
    const int sms = bq::device_sms();
    if (!sms) return BQ_ERR_CUDA;
    Args a;
    a.x = *x;
    a.wide = 1;
    // rows of 4-element vectors: the base pointers and, with several rows, the strides
    auto row_ok = [&](const void *p, int64_t stride, int es) {
        return !p || (bq::aligned_to(p, (uintptr_t)(4 * es)) && (x->rows == 1 || stride % 4 == 0));
    };
    a.wide = row_ok(x->y, x->y_stride, ey) && row_ok(x->gate, x->gate_stride, ey) &&
             row_ok(x->x, x->x_stride, ey) && row_ok(x->h, x->h_stride, eh) &&
             row_ok(x->h_out, x->h_out_stride, eh);
    a.wide_gain = bq::aligned_to(x->post, 16) && bq::aligned_to(x->pre, 16);
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
