// bq_attn_tcgen05.cuh -- the shared pages of a group of requests gone through once
// for all its query rows (the first pass of bq_paged_prefix_attention in
// include/bqgemv.h), for heads of up to 128 values.
//
// Mathematics.  For 128 query rows of one kv head at a time and tiles of 128 positions
// (64 over bf16 and Q8_0 caches): S = Q K^T, P = 2^(factor S - m), O = O + P V with a running reference
// m and sum l per row.  m follows the running maximum only when that has grown by
// more than 2^GROWTH, 2^8 or 2^4: weights are at most that then and O, which stays in
// tensor memory, is rescaled (by the row's own 2^(m_old - m)) in few tiles.
//
// A CTA takes a chunk of the positions for 128 rows.  Warps 0 to 3 and 4 to 7 are
// two streams: they take the even and the odd tiles, each with scores S (a column
// of tensor memory for each position) of its own, so that the tensor cores work for one stream while
// the other one computes its weights.  The streams hand the rows' references to one
// another and add into one O (up to 128 columns); the one that lets a reference grow
// rescales O.  Warp 8 brings K and V tiles into a ring in shared memory by tensor
// maps (pages that are whole groups of 8 slots; what is not there is filled with
// zeros), or warps 8 to 10 by 16-byte asynchronous copies (any page size and
// stride), in the swizzled rows of 128 bytes that the tensor cores read: K with
// positions as rows and head_dim contiguous, V the same bytes with the summed axis
// as rows.  One thread of warp 11 issues all products.  Queries are a first operand
// in tensor memory; the weights go back there in the columns of the scores that they
// come from, and are the first operand of the second product.  Over a Q8_0 cache
// warps 8 to 10, and those of warps 0 to 7 whose 32 rows are none of the group's, put
// codes times scales into parts on the way: the latter take 12 us off a call of 48 or 96
// rows of a kv head (30011 shared, 8 kv heads of 128).
//
// Bounds.  96 requests of 32801 shared, bf16, 32 over 8 heads of 128: 96 us, 535 TFLOP/s
// of scores and values counted once; products keep the tensor pipe busy for 44% (second
// and third parts of the weights two thirds of PV), the handing over of tiles of 64
// positions takes the rest, and 144 of 152 SMs have a chunk.  Over Q8_0 the putting into
// parts: 128 rows 4400 cycles a tile.
//
// Precision.  A query of the cache's type is used as it is, any other in QP 16-bit
// parts (fp16 2, after scaling the row by a power of two; bf16 3); weights are two
// parts of fp16, off by 2^-23, or three of bf16, 24 bits, as in the ordinary kernel
// (two of bf16, 17 bits, and O summed by the tensor core alone would do with bf16
// outputs but where terms cancel or a sum lies next to a rounding border: 0.7% of the
// outputs of 96 requests of 32801 shared were then not the nearest, 0.09% of an fp32
// form's).  Q8_0 codes times scales are two fp16 parts (below).  O is summed by the
// tensor core over some tiles and by fp32 additions over the chunk (FLUSH).
#pragma once

#include <cuda.h>  // CUtensorMap

#include <atomic>
#include <cmath>
#include <cstddef>

#include "bq_attn.h"

namespace bq {

constexpr int TC_ROWS = 128;
constexpr int TC_SOFTMAX_WARPS = 8, TC_COPY_WARPS = 3, TC_WARPS = 12;
constexpr int TC_MASKS = 8;        // tiles whose masks are kept
constexpr int TC_QBLOCK = TC_ROWS * 128;  // bytes of all rows' 64 values
constexpr int TC_COLUMNS = 512;      // of tensor memory, all of it

template <bool HALF, int QP, int NB, bool Q8>
struct TcShape {
    static constexpr int PP = HALF ? 2 : 3;  // parts of a weight
    // log2 of what a weight may be.  fp16 ones carry 2^SHIFT, so that they are up to 2^15, and
    // their parts keep 2^-25: 2^-32 of the reference's weight, or 2^-36 for fp32 queries, whose
    // outputs would show it where a position far above all others has little value (with
    // 2^-32 errors of up to 4e-5 of them, e^12 beside 1).  O is rescaled more often then, if
    // scores spread: 96 requests of 32801 shared, fp32 queries over fp16, scores of N(0, 1)
    // 122 us a call either way, of N(0, 9) 155 against 131.
    static constexpr int GROWTH = HALF && QP > 1 ? 4 : 8, SHIFT = HALF ? 15 - GROWTH : 0;
    // positions of a tile; bytes of its rows of 64 values; parts of a key or value
    static constexpr int TILE = Q8 || PP == 3 ? 64 : 128, BLOCK = TILE * 128, KP = Q8 ? 2 : 1;
    // The tensor core truncates when it adds to O: after some hundred positions that shows
    // in an fp32 output (chunks of 1800 positions: off by 4.4e-6 of it, fp32 sums 7e-7;
    // added up every 512 1.3e-6, every 256 8e-7), after thousands in a 16-bit one (fp16 1.3%
    // of the values not the nearest, with 512 0.4%, as fp32 sums leave; bf16, 32801 shared,
    // weights of three parts, with 512 0.12%, with 256 0.07%, fp32 sums 0.09%).  So O is
    // added up elsewhere in tensor memory, rounded to nearest, every FLUSH tiles, and
    // starts again.  fp16 heads of 128 then have their queries in shared memory: 96
    // requests of 32801 shared take 12 us more a call, with fp32 queries 31 more.
    static constexpr int FLUSH = (HALF && QP == 1 ? 512 : 256) / TILE;
    // columns of tensor memory: scores of two streams, O, its sum, and in the rest third
    // parts of the weights and, where there is room, queries (else these lie in shared memory)
    static constexpr int O = 2 * TILE, SUM = O + NB * 64, THIRD = 384, QUERIES = THIRD + (PP == 3 ? TILE : 0);
    static constexpr bool Q_TENSOR = SUM + NB * 64 <= THIRD && QUERIES + QP * NB * 32 <= TC_COLUMNS;
    static_assert(SUM + NB * 64 <= (PP == 3 ? THIRD : TC_COLUMNS));
    static constexpr int SLOT = KP * NB * BLOCK, Q_BYTES = Q_TENSOR ? 0 : QP * NB * TC_QBLOCK;
    static constexpr int LIMIT = 227 * 1024, MISC = 3 * 1024;
    // Q8_0: codes and scales on their way, RAW tiles of them, by groups of AT_ONCE rows; a
    // lane's 32 codes and a word with its scale
    static constexpr int RAW = 3, LANES = 2 * NB, AT_ONCE = 32 / LANES, GROUPS = TILE / AT_ONCE;
    static constexpr int MINE = (GROUPS + TC_COPY_WARPS - 1) / TC_COPY_WARPS;
    static constexpr int RAW_WARP = 32 * (32 + 4), RAW_TILE = 2 * GROUPS * RAW_WARP;
    static constexpr int RAW_BYTES = Q8 ? RAW * RAW_TILE : 0;
    static constexpr int most = (LIMIT - MISC - Q_BYTES - RAW_BYTES) / SLOT;
    static constexpr int SLOTS = most > 8 ? 8 : most;
    // Loads that are issued before the oldest is waited for.  A tile's keys are told as
    // arrived once the LAG loads behind them are issued, which takes slots that are free
    // again: with 3 of 6 the next keys waited for the values two tiles before (the pass
    // 126 us against 104), above SLOTS - 2 for themselves.
    static constexpr int LAG = SLOTS >= 8 ? 3 : 1;
    // (one CTA per SM: each takes all tensor memory)
    static constexpr int NEED = Q_BYTES + SLOTS * SLOT + RAW_BYTES + MISC, ALONE = 115 * 1024;
    static constexpr int SMEM = NEED > ALONE ? NEED : ALONE;
    static constexpr int OROW = NB * 64 + 4;  // floats of a row on its way out, in the ring's place
    static_assert(SLOTS >= 4 && LAG >= 1 && LAG <= SLOTS - 2);
    static_assert(TC_ROWS * OROW * 4 <= SLOTS * SLOT);
    static_assert(2 * (SMEM + 1024) > 228 * 1024 && SMEM <= LIMIT);
    // a copying warp is at most SLOTS / 2 tiles past one whose values are in use
    static_assert(SLOTS / 2 + 1 < TC_MASKS);
};

struct TcArgs {
    AttnArgs a;
    int box;        // positions of a copy by tensor map: the largest power of two that divides
                    // a page, 8 to 128; 0: copies of 16 bytes
    int heads_first;   // of the maps' axes: heads lie closer than slots
    int hold;          // TcHold
    uint64_t wait_ns;  // how long a wait lasts at most
    CUtensorMap k, v;  // [pages][kv heads][slots][head_dim] ([slots][kv heads]), in boxes of 64 values by `box` slots
};

// Barriers that a launch can be told to hold (more arrivals than ever come), so that a test
// sees the waits run out: the kernel gives up, says so and returns.
enum TcHold {
    TC_HOLD_NONE, TC_HOLD_QUERIES, TC_HOLD_FULL, TC_HOLD_EMPTY, TC_HOLD_MASK, TC_HOLD_SCORES, TC_HOLD_WEIGHTS,
    TC_HOLD_REFERENCE, TC_HOLD_FLUSHED, TC_HOLD_END, TC_HOLD_KINDS
};

// shared memory behind the ring
struct TcMisc {
    uint64_t full[8], empty[8], mask_full[TC_MASKS], s_full[2], p_full[2][2], q_full, added[2], flushed, summed[2], o_full;
    uint64_t ref_full[2][4];     // by stream and warp of it
    uint32_t top_scale[2];       // bits of the chunk's largest Q8_0 scales, of keys and values
    alignas(16) uint8_t mask[TC_MASKS][16];  // positions of a tile that are there
    float ref[2][TC_ROWS];       // a row's reference after the stream's last tile
    float sum[2][TC_ROWS];       // of its weights; the largest query values before
    uint32_t tmem;
    uint32_t dead;  // a wait has run out
};
static_assert(sizeof(TcMisc) <= 3 * 1024 && offsetof(TcMisc, mask) % 16 == 0 && alignof(TcMisc) == 16);

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
// the same without waiting a while for it
__device__ __forceinline__ uint32_t barrier_test(uint64_t *b, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
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
// Waits for a phase of the barrier, for `ns` at most; false if that has run out here or
// in another thread of the CTA.  Lanes of a warp may be told differently: it votes
// before it goes by the answer.
static __device__ __noinline__ bool barrier_wait_long(uint64_t *b, uint32_t parity, volatile uint32_t *dead, uint64_t ns) {
    const uint64_t t0 = tc_nanoseconds();
    while (!barrier_try(b, parity)) {
        if (*dead) return false;
        if (tc_nanoseconds() - t0 > ns) {
            *dead = 1;
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ bool barrier_wait(uint64_t *b, uint32_t parity, volatile uint32_t *dead, uint64_t ns) {
    if (barrier_try(b, parity)) return true;
    return barrier_wait_long(b, parity, dead, ns);
}
// The end of what a CTA has under way, before its memory is another's: a tenth of a
// second at most, whoever has given up.
static __device__ __noinline__ void barrier_wait_end(uint64_t *b, uint32_t parity) {
    const uint64_t t0 = tc_nanoseconds();
    while (!barrier_try(b, parity) && tc_nanoseconds() - t0 < 100000000ull) {}
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

__device__ __forceinline__ void tc_load8(uint32_t at, uint32_t (&v)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ void tc_store8(uint32_t at, const uint32_t (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"r"(v[0]), "r"(v[1]),
                 "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(at)
                 : "memory");
}

// A matrix in shared memory in rows of 128 bytes swizzled over 8 rows: its place,
// the distance of 64-value blocks (where the rows are the summed axis) and of
// groups of 8 rows
__device__ __forceinline__ uint64_t tc_matrix(uint32_t at, int block) {
    return (uint64_t)(at >> 4 & 0x3fff) | (uint64_t)(block >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 |
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
__device__ __forceinline__ void tc_store16(uint32_t at, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
// Four int8 codes as two pairs of fp16: with b = code + 128 (the sign bit turned)
// 0x6400 | b is 1024 + b, a whole number that fp16 holds; less 1152 it is the code.
__device__ __forceinline__ uint2 tc_codes(uint32_t w) {
    uint2 o;
    w ^= 0x80808080u;
    const uint32_t lo = __byte_perm(w, 0x64646464u, 0x4140), hi = __byte_perm(w, 0x64646464u, 0x4342);
    asm("sub.f16x2 %0, %1, %2;" : "=r"(o.x) : "r"(lo), "r"(0x64806480u));
    asm("sub.f16x2 %0, %1, %2;" : "=r"(o.y) : "r"(hi), "r"(0x64806480u));
    return o;
}
// true for one thread of the warp, the same each time
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one;
}
// the barrier's phase completes with all products issued so far
__device__ __forceinline__ void tc_commit(uint64_t *b) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(tc_shared(b))
                 : "memory");
}

__device__ __forceinline__ void tc_copy16(uint32_t dst, const void *src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
// a box of a tensor map into shared memory, zeros where it is outside; the barrier
// counts its bytes
__device__ __forceinline__ void tc_copy_box(uint32_t dst, const CUtensorMap *map, int x, int y, int z, int page,
                                            uint64_t *b) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(page), "r"(tc_shared(b))
        : "memory");
}
__device__ __forceinline__ void barrier_arrive_bytes(uint64_t *b, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(tc_shared(b)), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void tc_copy4(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
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

// pairs of fp32 values, two operations an instruction
__device__ __forceinline__ uint64_t pair_of(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 pair_values(uint64_t p) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p));
    return r;
}
__device__ __forceinline__ uint64_t pair_fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t pair_add(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t pair_less(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// the pair as two pairs of 16-bit numbers that add up to it
template <bool HALF>
__device__ __forceinline__ void pair_parts(uint64_t p, uint32_t &high, uint32_t &low) {
    const float2 v = pair_values(p);
    float2 h;
    if constexpr (HALF) {
        high = F16::down2(v.x, v.y);
        h = F16::up2(high);
    } else {
        high = BF16::down2(v.x, v.y);
        h = BF16::up2(high);
    }
    const float2 rest = pair_values(pair_less(p, pair_of(h.x, h.y)));
    low = HALF ? F16::down2(rest.x, rest.y) : BF16::down2(rest.x, rest.y);
}
// three that do
template <bool HALF>
__device__ __forceinline__ void pair_parts(uint64_t p, uint32_t &high, uint32_t &middle, uint32_t &low) {
    static_assert(!HALF);
    const float2 v = pair_values(p);
    high = BF16::down2(v.x, v.y);
    const float2 h = BF16::up2(high);
    pair_parts<HALF>(pair_less(p, pair_of(h.x, h.y)), middle, low);
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
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

template <bool HALF, int QP, int NB, bool Q8>
__global__ void __launch_bounds__(TC_WARPS * 32, 1)
    prefix_kernel(const __grid_constant__ TcArgs args, unsigned int *status) {
    using S = TcShape<HALF, QP, NB, Q8>;
    constexpr int TILE = S::TILE, BLOCK = S::BLOCK, FLUSH = S::FLUSH;
    const AttnArgs &a = args.a;
    constexpr int SLOTS = S::SLOTS, LAG = S::LAG;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *q_s = smem, *ring = smem + S::Q_BYTES;
    TcMisc &misc = *reinterpret_cast<TcMisc *>(ring + SLOTS * S::SLOT + S::RAW_BYTES);
    volatile uint32_t *dead = &misc.dead;
    const uint64_t limit = args.wait_ns;
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
    if (begin >= end || first_row >= group_rows) return;
    const int D16 = (D + 15) & ~15;
    // Q8_0: softmax warps whose 32 rows are none of the group's put codes into parts instead
    const int quads = Q8 ? min(4, (group_rows - first_row + 31) / 32) : 4;  // warps of a stream with rows
    const int copiers = TC_COPY_WARPS + 2 * (4 - quads);
    const bool softmax = warp < TC_SOFTMAX_WARPS && (!Q8 || (warp & 3) < quads);
    auto softmax_sync = [&] {
        if constexpr (Q8) asm volatile("bar.sync 1, %0;" ::"r"(64 * quads) : "memory");
        else asm volatile("bar.sync 1, 256;" ::: "memory");
    };

    // ---- barriers and tensor memory, while the kernel before ends ----
    if (tid == 0) {
        const int copying = Q8 ? copiers : args.box ? 1 : TC_COPY_WARPS;
        auto held = [&](TcHold which) { return args.hold == which ? 1 << 16 : 0; };
        for (int i = 0; i < SLOTS; ++i) {
            barrier_init(&misc.full[i], copying + (i ? 0 : held(TC_HOLD_FULL)));
            barrier_init(&misc.empty[i], 1 + (i ? 0 : held(TC_HOLD_EMPTY)));
        }
        for (int i = 0; i < TC_MASKS; ++i) barrier_init(&misc.mask_full[i], copying + (i ? 0 : held(TC_HOLD_MASK)));
        for (int i = 0; i < 2; ++i) {
            barrier_init(&misc.s_full[i], 1 + held(TC_HOLD_SCORES));
            for (int k = 0; k < 2; ++k) barrier_init(&misc.p_full[i][k], quads + (k ? held(TC_HOLD_WEIGHTS) : 0));
            for (int k = 0; k < 4; ++k) barrier_init(&misc.ref_full[i][k], 1 + (k ? 0 : held(TC_HOLD_REFERENCE)));
        }
        barrier_init(&misc.q_full, 2 * quads + held(TC_HOLD_QUERIES));
        for (int i = 0; i < 2; ++i) {
            barrier_init(&misc.added[i], 1);
            barrier_init(&misc.summed[i], quads);
        }
        barrier_init(&misc.flushed, quads + held(TC_HOLD_FLUSHED));
        barrier_init(&misc.o_full, 1 + held(TC_HOLD_END));
        misc.dead = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == TC_WARPS - 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc_shared(&misc.tmem)),
                     "n"(TC_COLUMNS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        tc_fence_before();
        if (lane < 2 && args.box)
            asm volatile("prefetch.tensormap [%0];" ::"l"(lane ? &args.v : &args.k) : "memory");
    }
    pdl_wait();
    pdl_launch_dependents();
    // the first request that holds the shared pages: its table row tells them
    int owner = 0x7fffffff;
    const int most = a.x.table_width * page;
    for (int i = first + lane; i < end_request && owner == 0x7fffffff; i += 32)
        if (attn_sees(attn_clamped(a.x.lens[i], most), R, common)) owner = i;
    owner = __reduce_min_sync(~0u, owner);
    // (without one nobody reads these partial results)
    const int tiles = owner == 0x7fffffff ? 0 : (end - begin + TILE - 1) / TILE;
    // Q8_0: keys and values go into two fp16 parts.  The chunk's largest scale brings the
    // largest possible value to [2^14, 2^15): nothing overflows, and what is down to
    // 2^-29 of it keeps a second part in fp16's range.
    [[maybe_unused]] const int *row_table = a.x.table + (tiles ? owner : 0) * a.x.table_stride;
    [[maybe_unused]] float by_keys = 1.0f, by_values = 1.0f;      // what the parts are to be multiplied by
    [[maybe_unused]] float of_keys = 1.0f, of_values = 1.0f;      // and were
    // element offset of position p, -1 where there is nothing to read
    [[maybe_unused]] auto offset_of = [&](int p, int entry) {
        if (entry < 0 || entry >= a.c.pages) return -1ll;
        const uint32_t in_page = (uint32_t)p - a.page.div((uint32_t)p) * a.page.d;
        return (long long)(entry * a.c.page_stride + in_page * a.c.slot_stride + (long long)h * a.c.head_stride);
    };
    if constexpr (Q8) {
        if (tid < 2) misc.top_scale[tid] = 0;
        __syncthreads();
        uint32_t top[2] = {0, 0};
        // (positions to threads, so that few loads wait for one another: with scales to
        // threads this took a third of the pass)
        const int blocks = D >> 5, last = tiles ? end : begin;
        for (int p0 = begin + tid; p0 < last; p0 += 4 * TC_WARPS * 32) {
            long long at[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int p = p0 + u * TC_WARPS * 32;
                at[u] = p < last ? offset_of(p, row_table[a.page.div((uint32_t)p)]) : -1;
            }
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int j = 0; j < 2 * NB; ++j) {
                    if (at[u] < 0 || j >= blocks) continue;
                    const uint32_t k = static_cast<const uint16_t *>(a.c.k_scale)[(at[u] >> 5) + j] & 0x7fffu;
                    const uint32_t v = static_cast<const uint16_t *>(a.c.v_scale)[(at[u] >> 5) + j] & 0x7fffu;
                    if (k < 0x7c00u) top[0] = max(top[0], k);  // (the finite ones: ordered as their bits)
                    if (v < 0x7c00u) top[1] = max(top[1], v);
                }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            top[k] = __reduce_max_sync(~0u, top[k]);
            if (lane == 0) atomicMax(&misc.top_scale[k], top[k]);
        }
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc.tmem;
    if constexpr (Q8) {
        auto power = [](uint32_t bits) {  // 127 scale 2^power is in [2^14, 2^15), or smaller
            const float top = 127.0f * __half2float(__ushort_as_half((unsigned short)bits));
            return top == 0.0f ? 0 : 14 - ((int)(__float_as_uint(top) >> 23) - 127);
        };
        const int pk = power(misc.top_scale[0]), pv = power(misc.top_scale[1]);
        by_keys = ldexpf(1.0f, -pk), by_values = ldexpf(1.0f, -pv);
        of_keys = ldexpf(1.0f, pk), of_values = ldexpf(1.0f, pv);
    }

    if (tiles == 0) {
    } else if (Q8 && !softmax && warp < TC_SOFTMAX_WARPS + TC_COPY_WARPS) {
        // ---- Q8_0: 8 (16) rows to each warp in turn, a lane a scale's 32 codes; the next
        // tile's are on their way while one is put into parts ----
        if constexpr (Q8) {
            constexpr int LANES = S::LANES, AT_ONCE = S::AT_ONCE, GROUPS = S::GROUPS, MINE = S::MINE, RAW = S::RAW;
            const int cw = warp >= TC_SOFTMAX_WARPS ? warp - TC_SOFTMAX_WARPS
                                                    : TC_COPY_WARPS + (warp >> 2) * (4 - quads) + (warp & 3) - quads;
            const int mine = cw < GROUPS ? (GROUPS - cw + copiers - 1) / copiers : 0;  // groups of this warp
            const int part = lane % LANES, sub = lane / LANES;
            const bool inside = 32 * part < D;
            // the halves of the 32 codes in an order that keeps a warp's stores apart in the
            // banks: lanes of another 64-value block take the other half first
            const int turn = part >> 1 & 1;
            uint8_t *raw = ring + SLOTS * S::SLOT;
            auto place = [&](int t, int v, int q) {
                return raw + (t % RAW) * S::RAW_TILE + (v * GROUPS + cw + copiers * q) * S::RAW_WARP;
            };
            auto row_of = [&](int q) { return (cw + copiers * q) * AT_ONCE + sub; };
            auto entry_of = [&](int q, int t) {
                const int p = begin + t * TILE + row_of(q);
                return q < mine && t < tiles && p < end ? row_table[a.page.div((uint32_t)p)] : -1;
            };
            int entry[MINE];
            uint32_t odd = 0;    // likewise: the scale is the second half of its word
            uint32_t there = 0;  // bits of the rows that this lane looks up, MINE for each of 4 tiles
            static_assert(4 * MINE <= 32 && RAW < 4);
            auto ask = [&](int t) {  // tile t's codes and scales; zeros where there is nothing
                const uint32_t of_tile = ~(((1u << MINE) - 1) << (t % 4 * MINE));
                there &= of_tile, odd &= of_tile;
#pragma unroll
                for (int q = 0; q < MINE; ++q) {
                    if (q >= mine) break;
                    const int p = begin + t * TILE + row_of(q);
                    const bool in = t < tiles && p < end;
                    const long long off = in ? offset_of(p, entry[q]) : -1;
                    if (in && off < 0 && part == 0) atomicOr(status, BQ_DEVERR_PAGE);
                    if (off >= 0) there |= 1u << (t % 4 * MINE + q);
                    const bool has = off >= 0 && inside;
                    const long long at = has ? off + 32 * part : 0;
                    odd |= (uint32_t)(at >> 5 & 1) << (t % 4 * MINE + q);
#pragma unroll
                    for (int v = 0; v < 2; ++v) {
                        const uint8_t *codes = static_cast<const uint8_t *>(v ? a.c.v : a.c.k) + at;
                        const uint8_t *scale = static_cast<const uint8_t *>(v ? a.c.v_scale : a.c.k_scale) + (at >> 6) * 4;
                        const uint32_t to = tc_shared(place(t, v, q));
                        tc_copy16(to + 16 * lane, codes + 16 * turn, has);
                        tc_copy16(to + 512 + 16 * lane, codes + 16 * (turn ^ 1), has);
                        // (the word that holds the scale, or where the cache ends with it its half)
                        tc_copy4(to + 1024 + 4 * lane, scale, !has ? 0 : (at >> 5 & 1) ? 4 : 2);
                    }
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
#pragma unroll
                for (int q = 0; q < MINE; ++q) entry[q] = entry_of(q, t + 1);
            };
            bool ok = true;
#pragma unroll
            for (int q = 0; q < MINE; ++q) entry[q] = entry_of(q, 0);
#pragma unroll 1
            for (int t = 0; t < RAW - 1; ++t) ask(t);
            for (int t = 0; t < tiles && ok; ++t) {
                ask(t + RAW - 1);
                tc_copies_wait<RAW - 1>();  // (a lane reads what it has copied itself)
#pragma unroll 1
                for (int v = 0; v < 2; ++v) {
                    const int n = 2 * t + v, slot = n % SLOTS;
                    ok = ok && barrier_wait(&misc.empty[slot], (n / SLOTS & 1) ^ 1, dead, limit);
                    ok = __all_sync(~0u, ok);
                    if (!ok) break;
                    if (v == 0) {
#pragma unroll
                        for (int q = 0; q < MINE; ++q) {
                            const uint32_t live = __ballot_sync(~0u, there >> (t % 4 * MINE + q) & 1);
                            // a byte for 8 rows, a bit of it for each row's first lane
                            uint32_t bits = 0;
#pragma unroll
                            for (int r = 0; r < AT_ONCE; ++r) bits |= (live >> (r * LANES) & 1) << r;
                            if (lane < AT_ONCE / 8 && q < mine)
                                misc.mask[t % TC_MASKS][(cw + copiers * q) * (AT_ONCE / 8) + lane] =
                                    (uint8_t)(bits >> (8 * lane));
                        }
                        __syncwarp();
                        if (lane == 0) barrier_arrive(&misc.mask_full[t % TC_MASKS]);
                    }
                    const uint32_t to = tc_shared(ring) + slot * S::SLOT + (part >> 1) * BLOCK;
#pragma unroll
                    for (int q = 0; q < MINE; ++q) {
                        if (q >= mine) break;
                        const int row = row_of(q);
                        // (a power of two times an fp16 number; exact in fp32, and in fp16 unless so
                        // small beside the chunk's largest that nothing of it is left)
                        const uint8_t *from = place(t, v, q);
                        const uint32_t both = *reinterpret_cast<const uint32_t *>(from + 1024 + 4 * lane);
                        const float d = __half2float(__ushort_as_half((unsigned short)(both >> (16 * (odd >> (t % 4 * MINE + q) & 1))))) *
                                        (v ? of_values : of_keys);
                        const __half2 d2 = __float2half2_rn(d);
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            const uint4 c = *reinterpret_cast<const uint4 *>(from + 512 * half + 16 * lane);
                            const uint32_t word[4] = {c.x, c.y, c.z, c.w};
                            uint32_t high[8], low[8];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const uint2 f = tc_codes(word[i]);
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    const uint32_t u = e ? f.y : f.x;
                                    const __half2 x = *reinterpret_cast<const __half2 *>(&u);
                                    const __half2 hi = __hmul2(x, d2);
                                    const __half2 lo = __hfma2(x, d2, __hneg2(hi));
                                    high[2 * i + e] = *reinterpret_cast<const uint32_t *>(&hi);
                                    low[2 * i + e] = *reinterpret_cast<const uint32_t *>(&lo);
                                }
                            }
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const int piece = 4 * (part & 1) + 2 * (turn ^ half) + i;
                                const uint32_t at = to + row * 128 + ((piece ^ (row & 7)) << 4);
                                tc_store16(at, high[4 * i], high[4 * i + 1], high[4 * i + 2], high[4 * i + 3]);
                                tc_store16(at + NB * BLOCK, low[4 * i], low[4 * i + 1], low[4 * i + 2], low[4 * i + 3]);
                            }
                        }
                    }
                    fence_async_proxy();
                    __syncwarp();
                    if (lane == 0) barrier_arrive(&misc.full[slot]);
                }
            }
            tc_copies_wait<0>();
        }
    } else if (warp == TC_SOFTMAX_WARPS && args.box) {
        // ---- copies by tensor maps: K and V of each tile in turn; lane j looks up the
        // tile's rows 8 j to 8 j + 7 (pages are whole groups of 8) ----
        auto entry_of = [&](int t) { return lane < TILE / 8 && t < end ? row_table[a.page.div((uint32_t)t)] : -1; };
        int entry = entry_of(begin + 8 * lane);
        const bool starts = lane < TILE / 8 && 8 * lane % args.box == 0;  // a box
        bool ok = true;
        int issued = 0;  // loads
        for (int t = 0; t < tiles && ok; ++t) {
            const int p = begin + t * TILE + 8 * lane;
            const bool in = lane < TILE / 8 && p < end, live = in && entry >= 0 && entry < a.c.pages;
            if (in && !live) atomicOr(status, BQ_DEVERR_PAGE);
            const int from = live ? entry : (int)a.c.pages;  // (outside the tensor: zeros)
            const int slot_of = live ? p - (int)a.page.div((uint32_t)p) * page : 0;
            entry = entry_of(p + TILE);
            for (int v = 0; v < 2; ++v) {
                const int n = 2 * t + v, slot = n % SLOTS;
                ok = __all_sync(~0u, barrier_wait(&misc.empty[slot], (n / SLOTS & 1) ^ 1, dead, limit));
                if (!ok) break;
                if (lane == 0) barrier_arrive_bytes(&misc.full[slot], S::SLOT);
                if (v == 0 && lane < TILE / 8) misc.mask[t % TC_MASKS][lane] = live ? 255 : 0;
                __syncwarp();
                if (v == 0 && lane == 0) barrier_arrive(&misc.mask_full[t % TC_MASKS]);
                if (starts) {
                    const uint32_t to = tc_shared(ring) + slot * S::SLOT + lane * 1024;
#pragma unroll
                    for (int b = 0; b < NB; ++b)
                        tc_copy_box(to + b * BLOCK, v ? &args.v : &args.k, 64 * b, args.heads_first ? h : slot_of,
                                    args.heads_first ? slot_of : h, from, &misc.full[slot]);
                }
                ++issued;
            }
        }
        if (!ok)  // (else the products have read them all)
            for (int n = max(0, issued - SLOTS); n < issued; ++n)
                barrier_wait_end(&misc.full[n % SLOTS], n / SLOTS & 1);
        __syncwarp();
    } else if (warp >= TC_SOFTMAX_WARPS && warp < TC_SOFTMAX_WARPS + TC_COPY_WARPS) {
        // ---- copies of 16 bytes (none where tensor maps do them): K and V of each tile in
        // turn, every third 8 rows by each warp ----
        constexpr int GROUPS = TILE / 8, MINE = (GROUPS + TC_COPY_WARPS - 1) / TC_COPY_WARPS;  // of 8 rows
        const int cw = warp - TC_SOFTMAX_WARPS;
        const long long head_off = (long long)h * a.c.head_stride;
        // rows that this lane looks up: of this warp's groups 0 to 3, and of 4 and 5
        auto row_at = [&](int k) { return 8 * (cw + TC_COPY_WARPS * (4 * k + (lane >> 3))) + (lane & 7); };
        auto entry_of = [&](int row, int t) { return row < TILE && t < end ? row_table[a.page.div((uint32_t)t)] : -1; };
        int entry[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) entry[k] = entry_of(row_at(k), begin + row_at(k));
        constexpr int PIECES = 8 * NB, AT_ONCE = 32 / PIECES, TURNS = 8 / AT_ONCE;  // of a row; rows at a time
        const int piece = lane % PIECES, sub = lane / PIECES;
        const bool there = piece < D16 / 8, inside = 8 * piece < D;
        // a group's rows lie one behind the other where pages are whole groups
        const bool in_line = page % 8 == 0;
        const long long hop = 2 * AT_ONCE * a.c.slot_stride;  // bytes from turn to turn
        const long long lane_at = 2 * sub * a.c.slot_stride + 16 * piece;
        const uint32_t ring_at = tc_shared(ring) + (piece >> 3) * BLOCK + sub * 128;
        uint32_t turn_at[TURNS];  // a row's place in its group of 8, swizzled
#pragma unroll
        for (int i = 0; i < TURNS; ++i)
            turn_at[i] = i * AT_ONCE * 128 + (((piece & 7) ^ ((i * AT_ONCE + sub) & 7)) << 4);
        auto arrived = [&](int n) {  // load n is complete: the products may read it
            fence_async_proxy();
            __syncwarp();
            if (lane == 0) barrier_arrive(&misc.full[n % SLOTS]);
        };
        bool ok = true;
        for (int t = 0; t < tiles && ok && !args.box; ++t) {
            long long off[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int p = begin + t * TILE + row_at(k);
                off[k] = -1;
                if (row_at(k) < TILE && p < end) {
                    if (entry[k] >= 0 && entry[k] < a.c.pages) {
                        const uint32_t in_page = (uint32_t)p - a.page.div((uint32_t)p) * a.page.d;
                        off[k] = entry[k] * a.c.page_stride + in_page * a.c.slot_stride + head_off;
                    } else {
                        atomicOr(status, BQ_DEVERR_PAGE);
                    }
                }
                entry[k] = entry_of(row_at(k), p + TILE);
            }
            uint32_t live[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) live[k] = __ballot_sync(~0u, off[k] >= 0);
            for (int v = 0; v < 2; ++v) {
                const int n = 2 * t + v, slot = n % SLOTS;
                ok = __all_sync(~0u, barrier_wait(&misc.empty[slot], (n / SLOTS & 1) ^ 1, dead, limit));
                if (!ok) break;
                // (after the wait: the masks of TC_MASKS tiles before are not in use any more)
                if (v == 0) {
                    const int of = cw + TC_COPY_WARPS * lane;
                    if (lane < MINE && of < GROUPS)
                        misc.mask[t % TC_MASKS][of] = (uint8_t)((lane < 4 ? live[0] : live[1]) >> (8 * (lane & 3)));
                    __syncwarp();
                    if (lane == 0) barrier_arrive(&misc.mask_full[t % TC_MASKS]);
                }
                const uint8_t *plane = static_cast<const uint8_t *>(v ? a.c.v : a.c.k);
#pragma unroll
                for (int q = 0; q < MINE; ++q) {
                    if (q == MINE - 1 && cw + TC_COPY_WARPS * q >= GROUPS) break;
                    const uint32_t to = ring_at + slot * S::SLOT + (cw + TC_COPY_WARPS * q) * 1024;
                    const uint32_t bits = live[q >> 2] >> (8 * (q & 3)) & 255;
                    if (bits == 255 && in_line) {
                        const long long o = __shfl_sync(~0u, off[q >> 2], 8 * (q & 3));
                        const uint8_t *src = plane + 2 * o + lane_at;
                        if (there) {
#pragma unroll
                            for (int i = 0; i < TURNS; ++i)
                                tc_copy16(to + turn_at[i], inside ? src + i * hop : plane, inside);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < TURNS; ++i) {
                            const long long o = __shfl_sync(~0u, off[q >> 2], 8 * (q & 3) + i * AT_ONCE + sub);
                            const bool has = o >= 0 && inside;
                            if (there) tc_copy16(to + turn_at[i], has ? plane + 2 * o + 16 * piece : plane, has);
                        }
                    }
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
                if (n >= LAG) {
                    tc_copies_wait<LAG>();
                    arrived(n - LAG);
                }
            }
        }
        tc_copies_wait<0>();
        if (ok && !args.box)
            for (int n = max(0, 2 * tiles - LAG); n < 2 * tiles; ++n) arrived(n);
    } else if (warp == TC_WARPS - 1) {
        // ---- products: the warp waits, one of its threads issues.  (The addresses are the
        // warp's, in uniform registers, and the steps unrolled: one thread that worked them
        // out in a loop took 97 cycles a step, of which the tensor cores need 64.) ----
        constexpr uint32_t SHAPE = 1u << 4 | (HALF ? 0u : 1u) << 7 | (HALF ? 0u : 1u) << 10 | (TC_ROWS >> 4) << 24;
        constexpr uint32_t qk_shape = SHAPE | (TILE >> 3) << 17;
        const uint32_t pv_shape = SHAPE | 1u << 16 | (uint32_t)(D16 >> 3) << 17;
        const uint64_t q_m = tc_matrix(tc_shared(q_s), TC_QBLOCK), ring_m = tc_matrix(tc_shared(ring), BLOCK);
        const int steps = D16 / 16;
        bool ok = __all_sync(~0u, barrier_wait(&misc.q_full, 0, dead, limit));
        // load n = 2 t of K, 2 t + 1 of V: in slot n % SLOTS, counted along
        int k_slot = 0, v_slot = 1;
        uint32_t k_phase = 0, v_phase = 0;
        auto next = [](int &slot, uint32_t &phase) {
            slot += 2;
            if (slot >= SLOTS) slot -= SLOTS, phase ^= 1;
        };
        auto waits = [&](uint64_t *b, uint32_t phase) {
            ok = ok && barrier_wait(b, phase, dead, limit);
            ok = __all_sync(~0u, ok);
        };
        auto scores = [&](int t) {  // S = Q K^T of tile t, smallest parts first; by the elected thread
            const uint64_t k_m = ring_m + k_slot * (S::SLOT >> 4);
            const uint32_t d = tmem + (t & 1) * TILE;
            // (the product of two second parts is below what either leaves out)
#pragma unroll
            for (int kp = S::KP - 1; kp >= 0; --kp)
#pragma unroll
                for (int p = kp ? 0 : QP - 1; p >= 0; --p)
#pragma unroll
                    for (int k = 0; k < 4 * NB; ++k) {
                        if (k >= steps) break;
                        const uint64_t keys = k_m + (kp * NB + (k >> 2)) * (BLOCK >> 4) + (k & 3) * 2;
                        const bool add = kp < S::KP - 1 || p < (kp ? 0 : QP - 1) || k;
                        if constexpr (S::Q_TENSOR)
                            tc_product_tensor(d, tmem + S::QUERIES + p * NB * 32 + 8 * k, keys, qk_shape, add);
                        else
                            tc_product_shared(d, q_m + (p * NB + (k >> 2)) * (TC_QBLOCK >> 4) + (k & 3) * 2, keys, qk_shape,
                                              add);
                    }
            tc_commit(&misc.empty[k_slot]);
            tc_commit(&misc.s_full[t & 1]);
        };
        for (int t = 0; t < 2 && t < tiles && ok; ++t) {
            waits(&misc.full[k_slot], k_phase);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) scores(t);
            __syncwarp();
            next(k_slot, k_phase);
        }
        const uint32_t o = tmem + S::O;
        // half of tile t's positions, 16 a step: 8 columns of a weight part; 32 columns
        // hold both parts of 32 positions
        auto output = [&](int t, int half) {
            const uint64_t v_m = ring_m + v_slot * (S::SLOT >> 4);
            const uint32_t w = tmem + (t & 1) * TILE;
            const bool goes_on = t % FLUSH != 0;  // O has something of this sum
            constexpr int STEPS = TILE / 32;
#pragma unroll
            for (int k = STEPS * half; k < STEPS * half + STEPS; ++k) {
                const uint32_t high = w + 32 * (k >> 1) + 8 * (k & 1);
                const uint64_t values = v_m + k * (2048 >> 4);
                if constexpr (S::PP == 3)
                    tc_product_tensor(o, tmem + S::THIRD + (t & 1) * (TILE / 2) + 8 * k, values, pv_shape, k || goes_on);
                tc_product_tensor(o, high + 16, values, pv_shape, S::PP == 3 || k || goes_on);
                if constexpr (Q8) tc_product_tensor(o, high, values + (NB * BLOCK >> 4), pv_shape, true);
                tc_product_tensor(o, high, values, pv_shape, true);
            }
        };
        for (int t = 0; t < tiles && ok; ++t) {
            const int s = t & 1;
            const bool more = t + 2 < tiles;
            uint64_t *keys = more ? &misc.full[k_slot] : &misc.full[v_slot];
            const uint32_t keys_phase = more ? k_phase : v_phase;
            const uint32_t there = barrier_test(&misc.full[v_slot], v_phase) & (Q8 || barrier_test(keys, keys_phase)) &
                                   barrier_test(&misc.p_full[s][0], t >> 1 & 1);
            if (!__all_sync(~0u, there)) {
                waits(&misc.full[v_slot], v_phase);
                if (!Q8) waits(keys, keys_phase);
                waits(&misc.p_full[s][0], t >> 1 & 1);
            }
            if (t && t % FLUSH == 0) waits(&misc.flushed, (t / FLUSH - 1) & 1);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) output(t, 0);
            __syncwarp();
            if (!__all_sync(~0u, barrier_test(&misc.p_full[s][1], t >> 1 & 1))) waits(&misc.p_full[s][1], t >> 1 & 1);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
                output(t, 1);
                tc_commit(&misc.empty[v_slot]);
                tc_commit(&misc.added[s]);
                if (!Q8 && more) scores(t + 2);
            }
            __syncwarp();
            // Q8_0: with 5 slots those keys take the place of the values before, and are put
            // into parts while the products above run
            if (Q8 && more) {
                waits(keys, keys_phase);
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) scores(t + 2);
                __syncwarp();
            }
            next(v_slot, v_phase);
            next(k_slot, k_phase);
        }
        // the end of all products; nothing is in flight when the tensor memory is given back
        if (elect_one()) tc_commit(&misc.o_full);
        __syncwarp();
        barrier_wait_end(&misc.o_full, 0);
        __syncwarp();
    } else {
        const int s = warp >> 2, i = 32 * (warp & 3) + lane;  // stream and row of this thread
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const int es = a.x.dtype == BQ_F32 ? 4 : 2;
        const bool wide = a.x.q_row_stride % 4 == 0 && a.x.q_head_stride % 4 == 0 &&
                          (reinterpret_cast<uintptr_t>(a.x.q) & (4 * es - 1)) == 0;
        // the row carries the scale's sign (and zero), so that a larger product is a
        // larger score
        const float sign = a.scale_log2 > 0.0f ? 1.0f : a.scale_log2 < 0.0f ? -1.0f : 0.0f;
        const float size = sign == 0.0f ? 1.0f : fabsf(a.scale_log2);
        auto read = [&](int gr, int d, float(&x)[4]) {  // 4 values of a query row of the group
            x[0] = x[1] = x[2] = x[3] = 0.0f;
            if (gr >= group_rows || d >= D) return;
            const int row = (int)a.group.div((uint32_t)gr), head = h * G + gr - row * G;
            const long long at = ((long long)first * R + row) * a.x.q_row_stride + head * a.x.q_head_stride + d;
            if (a.x.dtype == BQ_F32) load_n<F32, 4>((const float *)a.x.q + at, wide, x);
            else if (a.x.dtype == BQ_F16) load_n<F16, 4>((const __half *)a.x.q + at, wide, x);
            else load_n<BF16, 4>((const __nv_bfloat16 *)a.x.q + at, wide, x);
        };
        // powers of two that bring the largest of a row to [2^14, 2^15), as in the ordinary kernel
        struct Scaling {
            float a, b, factor;
        };
        auto scaling = [&](float top) {
            int ex = (int)((__float_as_uint(top) >> 23) & 0xff) - 127;
            if (top < 1.1754944e-38f || ex == 128) ex = 14;  // zero, subnormal or not finite: as it is
            const int up = 14 - ex;
            return Scaling{ldexpf(1.0f, up / 2), ldexpf(1.0f, up - up / 2),
                           size * ldexpf(1.0f, -(up / 2)) * ldexpf(1.0f, -(up - up / 2))};
        };
        constexpr bool SCALED = HALF && (QP > 1 || Q8);
        float factor;
        if constexpr (S::Q_TENSOR) {
            // ---- queries into tensor memory, a row to a thread, half of its values to each
            // stream's threads ----
            constexpr int EACH = NB * 32;  // values of this thread
            float x[EACH / 4][4], top = 0.0f;
#pragma unroll
            for (int k = 0; k < EACH / 4; ++k) {
                read(first_row + i, s * EACH + 4 * k, x[k]);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[k][e] *= sign;
                    if constexpr (SCALED) top = fmaxf(top, fabsf(x[k][e]));
                }
            }
            factor = size;
            Scaling by = {1.0f, 1.0f, size};
            if constexpr (SCALED) {
                misc.sum[s][i] = top;
                softmax_sync();
                by = scaling(fmaxf(misc.sum[0][i], misc.sum[1][i]));
                factor = by.factor;
            }
#pragma unroll
            for (int p = 0; p < QP; ++p)
#pragma unroll
                for (int k0 = 0; k0 < EACH / 4; k0 += 4) {
                    uint32_t w[8];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        float(&y)[4] = x[k0 + k];
                        if (SCALED && p == 0) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) y[e] = y[e] * by.a * by.b;
                        }
                        w[2 * k] = tc_part<HALF>(y[0], y[1]);
                        w[2 * k + 1] = tc_part<HALF>(y[2], y[3]);
                    }
                    tc_store8(tmem + lanes + S::QUERIES + p * NB * 32 + s * (EACH / 2) + 2 * k0, w);
                }
            tc_wait_store();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) barrier_arrive(&misc.q_full);
        } else {
            // ---- queries into shared memory, 16 rows to a warp ----
            const int d = 4 * lane;
            constexpr int EACH = TC_ROWS / TC_SOFTMAX_WARPS;
            float all[EACH][4];  // all rows' values on their way at once
#pragma unroll
            for (int k = 0; k < EACH; ++k) read(first_row + warp + TC_SOFTMAX_WARPS * k, d, all[k]);
#pragma unroll
            for (int k = 0; k < EACH; ++k) {
                const int r = warp + TC_SOFTMAX_WARPS * k;
                float(&x)[4] = all[k];
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] *= sign;
                if constexpr (SCALED) {
                    float top = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
                    const Scaling by = scaling(top);
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[e] = x[e] * by.a * by.b;
                    if (lane == 0) misc.sum[0][r] = by.factor;
                }
                const int piece = (lane & 15) >> 1;
                uint8_t *to = q_s + (lane >> 4) * TC_QBLOCK + r * 128 + ((piece ^ (r & 7)) << 4) + 8 * (lane & 1);
#pragma unroll
                for (int p = 0; p < QP; ++p) {
                    const uint2 w = make_uint2(tc_part<HALF>(x[0], x[1]), tc_part<HALF>(x[2], x[3]));
                    if (d < NB * 64) *reinterpret_cast<uint2 *>(to + p * NB * TC_QBLOCK) = w;
                }
            }
            fence_async_proxy();
            __syncwarp();
            if (lane == 0) barrier_arrive(&misc.q_full);
            factor = size;
            if constexpr (SCALED) {
                softmax_sync();  // factors of all rows
                factor = misc.sum[0][i];
            }
        }
        if constexpr (Q8) factor *= by_keys;
        // (above 0: what it multiplies may be minus infinity)
        factor = fmaxf(factor, 1.1754944e-38f);

        // ---- weights of this stream's tiles ----
        const uint32_t s_at = tmem + lanes + s * TILE, o_at = tmem + lanes + S::O;
        const uint32_t sum_at = tmem + lanes + S::SUM;
        float ref = -INFINITY, l = 0.0f;  // the reference that l belongs to
        bool ok = true;
        for (int t = s; t < tiles; t += 2) {
            ok = barrier_wait(&misc.mask_full[t % TC_MASKS], t / TC_MASKS & 1, dead, limit) &&
                 barrier_wait(&misc.s_full[s], t >> 1 & 1, dead, limit);
            if (!__all_sync(~0u, ok)) {
                ok = false;
                break;
            }
            tc_fence_after();
            uint32_t mask[TILE / 32], all = ~0u;
#pragma unroll
            for (int c = 0; c < TILE / 32; ++c) {
                mask[c] = reinterpret_cast<const uint32_t *>(misc.mask[t % TC_MASKS])[c];
                all &= mask[c];
            }
            if (all != ~0u) {  // positions that are not there: minus infinity
#pragma unroll 1
                for (int c = 0; c < TILE; c += 8) {
                    const uint32_t bits = misc.mask[t % TC_MASKS][c >> 3];
                    uint32_t o[8];
                    tc_load8(s_at + c, o);
                    tc_wait_load();
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (!(bits >> k & 1)) o[k] = 0xff800000u;
                    tc_store8(s_at + c, o);
                }
                tc_wait_store();
            }
            uint32_t x[2][32];
            float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            auto largest = [&](const uint32_t(&y)[32]) {
#pragma unroll
                for (int k = 0; k < 32; k += 2)
                    m[k / 2 & 3] = max3(m[k / 2 & 3], __uint_as_float(y[k]), __uint_as_float(y[k + 1]));
            };
            tc_load32(s_at, x[0]);
            tc_load32(s_at + 32, x[1]);
            tc_wait_load();
            largest(x[0]);
            if constexpr (TILE > 64) tc_load32(s_at + 64, x[0]);
            largest(x[1]);
            if constexpr (TILE > 64) {
                tc_load32(s_at + 96, x[1]);
                tc_wait_load();
                largest(x[0]);
                largest(x[1]);
            }
            const float top = fmaxf(max3(m[0], m[1], m[2]), m[3]) * factor;
            // the reference that the tile before left, the other stream's
            float was = -INFINITY;
            if (t) {
                ok = barrier_wait(&misc.ref_full[s ^ 1][warp & 3], (t - 1) >> 1 & 1, dead, limit);
                if (!__all_sync(~0u, ok)) {
                    ok = false;
                    break;
                }
                was = misc.ref[s ^ 1][i];
            }
            const bool grows = top > was + (float)S::GROWTH || (was == -INFINITY && top > was);
            const float now = grows ? top : was;
            misc.ref[s][i] = now;
            __syncwarp();
            if (lane == 0) barrier_arrive(&misc.ref_full[s][warp & 3]);
            if (t && __any_sync(~0u, grows)) {  // O of the tiles before, once it is there
                // (where it starts again with this tile, its sum once it is added there)
                const bool again = t % FLUSH == 0;
                // (A wait by parity must be at most one phase behind: the barriers are one to a
                // stream, or to every other sum, whose phase before is known to be over.)
                const int sums = t / FLUSH - 1;
                ok = again ? barrier_wait(&misc.summed[sums & 1], sums >> 1 & 1, dead, limit)
                           : barrier_wait(&misc.added[s ^ 1], (t - 1) >> 1 & 1, dead, limit);
                if (!__all_sync(~0u, ok)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const float alpha = grows ? tc_pow2(was - now) : 1.0f;
                auto rescale = [&](uint32_t at) {
#pragma unroll 1
                    for (int c = 0; c < D16; c += 8) {
                        uint32_t o[8];
                        tc_load8(at + c, o);
                        tc_wait_load();
#pragma unroll
                        for (int k = 0; k < 8; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
                        tc_store8(at + c, o);
                    }
                };
                if (!again) rescale(o_at);
                if (t >= FLUSH) rescale(sum_at);
            }
            if (ref != now) l *= tc_pow2(ref - now);
            ref = now;
            tc_load32(s_at, x[0]);
            const float shift = (float)S::SHIFT - (ref == -INFINITY ? 0.0f : ref);
            const uint64_t factors = pair_of(factor, factor), shifts = pair_of(shift, shift);
            uint64_t sum[2] = {0, 0};
            auto told = [&](int half) {  // half of the weights are in tensor memory
                tc_wait_store();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) barrier_arrive(&misc.p_full[s][half]);
            };
            auto weights = [&](const uint32_t(&y)[32], int c) {
                uint32_t w[32];
                [[maybe_unused]] uint32_t third[16];
#pragma unroll
                for (int k = 0; k < 32; k += 2) {
                    const float2 e = pair_values(
                        pair_fma(pair_of(__uint_as_float(y[k]), __uint_as_float(y[k + 1])), factors, shifts));
                    const uint64_t p = pair_of(tc_pow2(e.x), tc_pow2(e.y));
                    sum[k / 2 & 1] = pair_add(sum[k / 2 & 1], p);
                    if constexpr (S::PP == 3) pair_parts<HALF>(p, w[k / 2], w[16 + k / 2], third[k / 2]);
                    else pair_parts<HALF>(p, w[k / 2], w[16 + k / 2]);
                }
                if (c == TILE / 64) told(0);  // (its store has had this chunk's time)
                tc_store32(s_at + 32 * c, w);
                if constexpr (S::PP == 3) {
                    tc_store8(tmem + lanes + S::THIRD + s * (TILE / 2) + 16 * c, reinterpret_cast<uint32_t(&)[8]>(third[0]));
                    tc_store8(tmem + lanes + S::THIRD + s * (TILE / 2) + 16 * c + 8, reinterpret_cast<uint32_t(&)[8]>(third[8]));
                }
            };
#pragma unroll 1
            for (int c = 0; c < TILE / 32; c += 2) {  // (unrolled, the code outgrows the instruction cache)
                tc_wait_load();
                tc_load32(s_at + 32 * c + 32, x[1]);
                weights(x[0], c);
                tc_wait_load();
                if (TILE > 64 && c == 0) tc_load32(s_at + 64, x[0]);
                weights(x[1], c + 1);
            }
            told(1);
            const float2 l2 = pair_values(pair_add(sum[0], sum[1]));
            l += l2.x + l2.y;
            if ((t + 1) % FLUSH == 0 && t + 1 < tiles) {  // O to its sum, before it starts again
                ok = barrier_wait(&misc.added[s], t >> 1 & 1, dead, limit);
                if (!__all_sync(~0u, ok)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                // O into registers, and it may start again: the sum is not waited for
                uint32_t o[2 * NB][32];
#pragma unroll
                for (int c = 0; c < 2 * NB; ++c) tc_load32(o_at + 32 * c, o[c]);
                tc_wait_load();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) barrier_arrive(&misc.flushed);
                const bool first_time = t + 1 == FLUSH;
#pragma unroll
                for (int c = 0; c < 8 * NB; ++c) {
                    uint32_t u[8];
                    if (!first_time) {
                        tc_load8(sum_at + 8 * c, u);
                        tc_wait_load();
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float v = __uint_as_float(o[c / 4][8 * (c % 4) + e]);
                        u[e] = __float_as_uint(first_time ? v : v + __uint_as_float(u[e]));
                    }
                    tc_store8(sum_at + 8 * c, u);
                }
                tc_wait_store();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) barrier_arrive(&misc.summed[((t + 1) / FLUSH - 1) & 1]);
            }
        }

        // ---- the partial results, through the ring's place: nothing reads or fills it once
        // the last products are complete ----
        ok = ok && barrier_wait(&misc.o_full, 0, dead, limit);
        ok = __all_sync(~0u, ok);
        tc_fence_before();
        softmax_sync();  // (the one stream may still be at its sum)
        tc_fence_after();
        misc.ref[s][i] = ref, misc.sum[s][i] = l;
        // partial results of the ordinary kernel carry 2^ATTN_SHIFT_F16 over fp16 caches
        constexpr float LIKE = HALF ? (float)(1 << (ATTN_SHIFT_F16 - S::SHIFT)) : 1.0f;
        const float out = Q8 ? LIKE * by_values : LIKE;
        float *row = reinterpret_cast<float *>(ring) + i * S::OROW;
        for (int c = 8 * s; c < D16 && ok; c += 16) {
            uint32_t x[8];
            tc_load8(o_at + c, x);
            if (tiles > FLUSH) {
                uint32_t u[8];
                tc_load8(sum_at + c, u);
                tc_wait_load();
#pragma unroll
                for (int k = 0; k < 8; ++k) x[k] = __float_as_uint(__uint_as_float(x[k]) + __uint_as_float(u[k]));
            }
            tc_wait_load();
#pragma unroll
            for (int k = 0; k < 8; k += 4)
                *reinterpret_cast<float4 *>(row + c + k) =
                    make_float4(out * __uint_as_float(x[k]), out * __uint_as_float(x[k + 1]),
                                out * __uint_as_float(x[k + 2]), out * __uint_as_float(x[k + 3]));
        }
        softmax_sync();
        const long long unit = (((long long)g * a.max_chunks + ck) * KVH + h) * a.row_tiles + rt;
        if (s == 0 && first_row + i < group_rows) {
            // O belongs to the last tile's reference, which the other stream's sum may not
            const int last = (tiles - 1) & 1;
            const float top = misc.ref[last][i], other = misc.ref[last ^ 1][i];
            const float f = other == top ? 1.0f : tc_pow2(other - top);
            a.part_ml[unit * TC_ROWS + i] =
                make_float2(top, LIKE * (misc.sum[last][i] + (other == -INFINITY ? 0.0f : f * misc.sum[last ^ 1][i])));
        }
        if (4 * lane < D) {
            float *dst = a.part_o + unit * TC_ROWS * D + 4 * lane;
            const float *src = reinterpret_cast<const float *>(ring) + 4 * lane;
            for (int r = s * quads + (warp & 3); r < TC_ROWS && first_row + r < group_rows; r += 2 * quads)
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

template <bool HALF, int QP, int NB, bool Q8>
cudaError_t prefix_launch_of(const TcArgs &a, int grid, void *stream, unsigned int *status) {
    auto *kern = prefix_kernel<HALF, QP, NB, Q8>;
    constexpr int smem = TcShape<HALF, QP, NB, Q8>::SMEM;
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
template <bool HALF, int QP, bool Q8 = false>
cudaError_t prefix_launch(const TcArgs &a, int grid, void *stream, unsigned int *status) {
    return a.a.c.head_dim <= 64 ? prefix_launch_of<HALF, QP, 1, Q8>(a, grid, stream, status)
                              : prefix_launch_of<HALF, QP, 2, Q8>(a, grid, stream, status);
}

}  // namespace bq
