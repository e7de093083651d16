// bq_append.cu -- checks and launch of the append (bq_kv_append and
// bq_kv_append_norm in include/bqgemv.h; the kernel is bq_append.cuh).
#include <atomic>
#include <cmath>

#include "bq_append.cuh"

namespace {

BQ_STATUS_WORD(append)

// the status word's device address, looked up once per device
cudaError_t status_address(unsigned int **out) {
    static std::atomic<unsigned int *> addr[64];
    return bq::symbol_address(addr, g_status_append, out);
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

static bq_status append(const bq_kv_cache *cache, const bq_kv_append_args *x, const bq_kv_norm_args *norm, void *stream) {
    using bq::AppendArgs, bq::MAX_BATCH, bq::MAX_WARPS, bq::UNROLL, bq::warp_smem;
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
    if (norm && !(std::isfinite(norm->eps) && norm->eps >= 0.0f)) return BQ_ERR_SHAPE;
    if (x->tokens == 0) return BQ_OK;
    s = bq::check_cache_pointers(cache);
    if (s != BQ_OK) return s;
    if (!x->k || !x->v || !x->slots || (x->q && !x->q_out) || (x->freq && !x->positions)) return BQ_ERR_NULL;
    const void *typed[] = {x->k, x->v, x->q, x->q ? x->q_out : nullptr};
    for (const void *p : typed)
        if (!bq::aligned_to(p, (uintptr_t)es)) return BQ_ERR_ALIGN;
    if (!bq::aligned_to(x->slots, 8) || (x->freq && (!bq::aligned_to(x->freq, 8) || !bq::aligned_to(x->positions, 4))))
        return BQ_ERR_ALIGN;
    if (norm && (!bq::aligned_to(norm->q_gain, 4) || !bq::aligned_to(norm->k_gain, 4))) return BQ_ERR_ALIGN;
    const int sms = bq::device_sms();
    if (!sms) return BQ_ERR_CUDA;
    AppendArgs a;
    a.c = *cache;
    a.x = *x;
    a.n = norm ? *norm : bq_kv_norm_args{};
    if (!x->q) a.n.q_gain = nullptr;
    const bool normed = a.n.q_gain || a.n.k_gain;  // (gains NULL: the call without norms, bit for bit)
    a.inv_dim = 1.0f / (float)cache->head_dim;
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
    const int by_smem = 228 * 1024 / (a.smem + 2 * MAX_BATCH * 4 * gl * 8 + (normed ? 64 * gl : 0) + 1024 + 256);
    const long long fit = (long long)sms * (24 / a.warps < by_smem ? 24 / a.warps : by_smem);
    const long long each = (x->tokens * a.parts + fit - 1) / fit;
    a.batch = each < 1 ? 1 : each > MAX_BATCH ? MAX_BATCH : (int)each;
    const long long groups = (x->tokens + a.batch - 1) / a.batch;
    const long long most = (fit + a.parts - 1) / a.parts;
    const int grid = (int)(groups < most ? groups : most) * a.parts;
    unsigned int *status = nullptr;
    const cudaError_t e = status_address(&status);
    if (e != cudaSuccess) return bq::from_cuda_error(e);
    return bq::from_cuda_error(normed ? bq::append_normed(a, grid, stream, status)
                                      : bq::append_launch<false>(a, grid, stream, status));
}

extern "C" bq_status bq_kv_append(const bq_kv_cache *cache, const bq_kv_append_args *x, void *stream) {
    return append(cache, x, nullptr, stream);
}

extern "C" bq_status bq_kv_append_norm(const bq_kv_cache *cache, const bq_kv_append_args *x, const bq_kv_norm_args *norm,
                                       void *stream) {
    if (!norm) return BQ_ERR_NULL;
    return append(cache, x, norm, stream);
}
