// bq_cache.cuh -- shared by the kernels around the paged key-value cache and
// the block norms (bq_tables.cu, bq_append.cu, bq_attn.cuh, bq_norm.cu): typed
// loads and stores, division by a launch constant, programmatic launch.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "../../include/bqgemv.h"
#include "bq_internal.h"

namespace bq {

// Unsigned division of n < 2^31 by a divisor 1 <= d < 2^31 fixed at launch:
// q = n * m >> (31 + s) with s = ceil(log2 d), m = ceil(2^(31+s) / d).  m < 2^32
// and m*d - 2^(31+s) < d <= 2^s, so the error n * (m*d - 2^(31+s)) / (d * 2^(31+s))
// is below 1/d for every n < 2^31 and the quotient is exact.
struct FastDiv {
    uint32_t d, m, s;
    __host__ void set(uint32_t div) {
        d = div;
        s = 0;
        while ((1ull << s) < div) ++s;
        m = (uint32_t)(((1ull << (31 + s)) + div - 1) / div);
    }
    __host__ __device__ __forceinline__ uint32_t div(uint32_t n) const {
        return (uint32_t)(((uint64_t)n * m) >> (31 + s));
    }
};

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch_dependents() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Launch with programmatic dependent launch allowed: every kernel launched
// here executes pdl_wait before its first access to global memory.
// `cluster` > 1: CTAs per thread-block cluster.
template <typename... P, typename... A>
inline cudaError_t launch_pdl(void (*kern)(P...), dim3 grid, int threads, size_t smem, void *stream,
                              int cluster, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

// element types of activations as template tags; two of a 16-bit type at a time
struct F32 {
    using T = float;
    static __device__ __forceinline__ float up(float v) { return v; }
    static __device__ __forceinline__ float down(float v) { return v; }
};
struct F16 {
    using T = __half;
    static __device__ __forceinline__ float up(__half v) { return __half2float(v); }
    static __device__ __forceinline__ __half down(float v) { return __float2half_rn(v); }
    static __device__ __forceinline__ float2 up2(uint32_t w) {
        return __half22float2(*reinterpret_cast<const __half2 *>(&w));
    }
    static __device__ __forceinline__ uint32_t down2(float x, float y) {
        uint32_t w;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(y), "f"(x));
        return w;
    }
};
struct BF16 {
    using T = __nv_bfloat16;
    static __device__ __forceinline__ float up(__nv_bfloat16 v) { return __bfloat162float(v); }
    static __device__ __forceinline__ __nv_bfloat16 down(float v) { return __float2bfloat16_rn(v); }
    static __device__ __forceinline__ float2 up2(uint32_t w) {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
    static __device__ __forceinline__ uint32_t down2(float x, float y) {
        uint32_t w;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(y), "f"(x));
        return w;
    }
};

// N (4 or 8) consecutive elements by 16-byte (8-byte) accesses; the address is
// aligned to 4 elements of a 16-bit type for N = 4, else to 16 bytes
template <class E, int N>
__device__ __forceinline__ void load_wide(const typename E::T *p, float (&out)[N]) {
    if constexpr (sizeof(typename E::T) == 4) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const float4 v = reinterpret_cast<const float4 *>(p)[i];
            out[4 * i] = v.x, out[4 * i + 1] = v.y, out[4 * i + 2] = v.z, out[4 * i + 3] = v.w;
        }
    } else {
        uint32_t w[N / 2];
        if constexpr (N == 4) {
            const uint2 v = *reinterpret_cast<const uint2 *>(p);
            w[0] = v.x, w[1] = v.y;
        } else {
            const uint4 v = *reinterpret_cast<const uint4 *>(p);
            w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
        }
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const float2 f = E::up2(w[i]);
            out[2 * i] = f.x, out[2 * i + 1] = f.y;
        }
    }
}

template <class E, int N>
__device__ __forceinline__ void store_wide(typename E::T *p, const float (&in)[N]) {
    if constexpr (sizeof(typename E::T) == 4) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i)
            reinterpret_cast<float4 *>(p)[i] = make_float4(in[4 * i], in[4 * i + 1], in[4 * i + 2], in[4 * i + 3]);
    } else {
        uint32_t w[N / 2];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) w[i] = E::down2(in[2 * i], in[2 * i + 1]);
        if constexpr (N == 4)
            *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
        else
            *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// the same, element by element unless `wide`
template <class E, int N>
__device__ __forceinline__ void load_n(const typename E::T *p, bool wide, float (&out)[N]) {
    if (wide) {
        load_wide<E, N>(p, out);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) out[i] = E::up(p[i]);
    }
}
template <class E, int N>
__device__ __forceinline__ void store_n(typename E::T *p, bool wide, const float (&in)[N]) {
    if (wide) {
        store_wide<E, N>(p, in);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) p[i] = E::down(in[i]);
    }
}

// host-side argument checks
inline bool aligned_to(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline int dtype_bytes(int t) { return t == BQ_F32 ? 4 : t == BQ_F16 || t == BQ_BF16 ? 2 : 0; }
// (a failed call's error is taken off the thread, so that it is not found by a
// later, unrelated cudaGetLastError)
inline bq_status from_cuda_error(cudaError_t e) {
    if (e == cudaSuccess) return BQ_OK;
    cudaGetLastError();
    return BQ_ERR_CUDA;
}

// what bqgemv.h says of bq_kv_cache: shapes and strides, then pointers
inline bq_status check_cache_shape(const bq_kv_cache *c) {
    if (!c) return BQ_ERR_NULL;
    const bool q8 = c->type == BQ_Q8_0;
    if (!q8 && c->type != BQ_F16 && c->type != BQ_BF16) return BQ_ERR_QTYPE;
    const int step = q8 ? 32 : 8;
    if (c->head_dim < step || c->head_dim > 256 || c->head_dim % step) return BQ_ERR_SHAPE;
    if (c->kv_heads < 1 || c->kv_heads > 1024 || c->page_size < 1 || c->page_size > 65536 ||
        c->pages < 1 || c->pages > 0x7fffffffLL)
        return BQ_ERR_SHAPE;
    const int64_t mul = q8 ? c->head_dim : 8;
    const int64_t strides[3] = {c->page_stride, c->head_stride, c->slot_stride};
    for (int64_t s : strides)
        if (s < 0 || s > 0x7fffffffLL || s % mul) return BQ_ERR_SHAPE;
    return BQ_OK;
}
inline bq_status check_cache_pointers(const bq_kv_cache *c) {
    if (!c->k || !c->v) return BQ_ERR_NULL;
    if (!aligned_to(c->k, 16) || !aligned_to(c->v, 16)) return BQ_ERR_ALIGN;
    if (c->type == BQ_Q8_0) {
        if (!c->k_scale || !c->v_scale) return BQ_ERR_NULL;
        if (!aligned_to(c->k_scale, 8) || !aligned_to(c->v_scale, 8)) return BQ_ERR_ALIGN;
    }
    return BQ_OK;
}

// SMs of the current device, 0 on failure
int device_sms();

// the device address of a word, looked up once per device
inline cudaError_t symbol_address(std::atomic<unsigned int *> (&addr)[64], const unsigned int &symbol,
                                  unsigned int **out) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    unsigned int *p = addr[dev].load();
    if (!p) {
        e = cudaGetSymbolAddress(reinterpret_cast<void **>(&p), symbol);
        if (e != cudaSuccess) return e;
        addr[dev].store(p);
    }
    *out = p;
    return cudaSuccess;
}

}  // namespace bq

// a translation unit's status word and its reader
#define BQ_STATUS_WORD(NAME)                                                                       \
    static __device__ unsigned int g_status_##NAME = 0;                                            \
    static inline int read_status_##NAME(unsigned int *flags, int clear) {                         \
        cudaError_t e = cudaMemcpyFromSymbol(flags, g_status_##NAME, sizeof(unsigned int));        \
        if (e != cudaSuccess) return (int)e;                                                       \
        if (clear) {                                                                               \
            const unsigned int zero = 0;                                                           \
            e = cudaMemcpyToSymbol(g_status_##NAME, &zero, sizeof(unsigned int));                  \
        }                                                                                          \
        return (int)e;                                                                             \
    }
