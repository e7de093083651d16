// bq_pages.cu -- pages that requests share: block tables of a step with forks and
// counts (bq_kv_shared_tables), copies of pages in all layers (bq_kv_copy_pages)
// and compaction of the pool (bq_kv_compact), in include/bqgemv.h.
//
// The tables are one launch of one thread-block cluster, in phases between cluster
// barriers: scans of the requests (every CTA does them all, in its shared memory);
// then forked rows copied, popped pages written, counts raised and lowered, by
// atomics whose sums do not depend on their order; then, if pages are given up, the
// ones whose count has come to 0 claimed, each by its first release (an atomic
// minimum over the releases' indices, kept in the count itself as a negative
// number), the claims ranked by a scan over the releases, and pushed.  So nothing
// depends on the order of threads.  Bound by latency: a barrier is a few hundred ns,
// a phase one or two reads from L2 after one another.  24 requests with 15 forks 11 us,
// 1000 with 120 forks 33 us, the token rows' launch with it.
//
// Compaction ranks the pages by ballots and prefix sums over the pool (one cluster),
// then renumbers the tables over the whole GPU: 3000 pages 7 us, 200000 pages 20.
// Copies are bound by HBM: each thread has 64 bytes in flight, 16 KB per CTA and turn;
// 200 pages of 28 layers, 367 MB there and back, 113 us, 6.5 TB/s.
#include <atomic>

#include "bq_tables.cuh"

namespace {

BQ_STATUS_WORD(pages)

constexpr int THREADS = 1024, WARPS = THREADS / 32;
constexpr int CLUSTER = 8, CLUSTER_MOST = 16;  // CTAs
constexpr int CLAIM = -0x7fffffff - 1;  // count of a page that is given back: CLAIM + its first release

struct ShareArgs {
    bq_kv_tables t;
    bq_kv_sharing s;
    bq::FastDiv page;
};

__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
// a word of shared memory of another CTA of the cluster
__device__ __forceinline__ long long peer_word(const long long *at, uint32_t rank) {
    long long v;
    asm volatile("{\n\t.reg .b32 p;\n\tmapa.shared::cluster.u32 p, %1, %2;\n\tld.shared::cluster.s64 %0, [p];\n\t}"
                 : "=l"(v)
                 : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(at))), "r"(rank)
                 : "memory");
    return v;
}

// Sums that stop at 2^31 - 1, which is more than any pool, max_tokens or number of
// entries: a stopped sum decides as the true one does.
__device__ __forceinline__ uint32_t add_up(uint32_t a, uint32_t b) { return min(a + b, 0x7fffffffu); }

// exclusive prefix sums over the CTA's threads of K numbers each, and their totals
template <int K>
__device__ __forceinline__ void scan_threads(uint32_t (&v)[K], uint32_t (&total)[K], uint32_t (*scratch)[WARPS]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    uint32_t before[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t u = __shfl_up_sync(~0u, v[k], o);
            if (lane >= o) v[k] = add_up(v[k], u);
        }
        if (lane == 31) scratch[k][warp] = v[k];
        before[k] = __shfl_up_sync(~0u, v[k], 1);
        if (lane == 0) before[k] = 0;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
        uint32_t w = lane < warps ? scratch[k][lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t u = __shfl_up_sync(~0u, w, o);
            if (lane >= o) w = add_up(w, u);
        }
        total[k] = __shfl_sync(~0u, w, 31);
        const uint32_t others = __shfl_sync(~0u, w, (warp + 31) & 31);
        v[k] = add_up(before[k], warp ? others : 0);
    }
    __syncthreads();
}

__global__ void __launch_bounds__(THREADS) share_kernel(const __grid_constant__ ShareArgs a, int with_rows) {
    extern __shared__ int sm[];
    const int n = a.t.requests, tid = threadIdx.x, threads = blockDim.x;
    // per request: length before its rows, length asked, parent and marks, the page
    // that it copies; exclusive prefix sums
    int *base_s = sm, *want_s = base_s + n, *mark_s = want_s + n, *last_s = mark_s + n;
    int *asked = last_s + n, *rows = asked + n + 1, *gone = rows + n + 1, *joined = gone + n + 1, *copied = joined + n + 1;
    __shared__ uint32_t scratch[3][WARPS];
    __shared__ long long s_pushed;  // of this CTA
    __shared__ int s_given, s_refused;
    constexpr int CUT = 1 << 16, BAD = 1 << 17, SERVED = 1 << 18, PARENT = CUT - 1;
    bq::pdl_wait();
    if (!with_rows) bq::pdl_launch_dependents();
    const uint32_t rank = cluster_rank(), cluster = cluster_size();
    if (tid == 0) s_given = s_refused = 0;
    const long long most = (long long)a.t.table_width * a.t.page_size;
    const int count_in = *a.t.free_count, pool = a.t.pool;
    const int count = min(max(count_in, 0), pool);
    if (count != count_in && tid == 0 && rank == 0) atomicOr(&g_status_pages, BQ_DEVERR_POOL);
    auto pages = [&](int len) {
        const uint32_t q = a.page.div((uint32_t)len);
        return (int)(q + ((uint32_t)len - q * a.page.d != 0));
    };

    // ---- what each request starts from ----
    for (int b = tid; b < n; b += threads) {
        const int lo = a.t.lens[b], hi = a.t.new_lens[b];
        int p = a.s.parents ? a.s.parents[b] : -1;
        bool bad = lo < 0 || hi < 0 || lo > most || hi > most;
        int base = lo;
        if (p >= 0) {
            bad = bad || lo != 0 || p >= n || p == b;
            const int of = bad ? 0 : a.t.lens[p];
            bad = bad || of < 0 || of > most || a.s.parents[p] >= 0;
            if (!bad) base = min(of, hi);
        }
        if (bad || p < 0) p = -1;
        bool cut = false;  // the last page becomes its own
        int last = -1;
        if (!bad && hi > base && base > 0) {
            const int held = pages(base);
            if ((long long)held * a.t.page_size != base) {
                last = a.t.table[(long long)(p >= 0 ? p : b) * a.t.table_stride + held - 1];
                if (last < 0 || last >= pool) {
                    if (rank == 0) atomicOr(&g_status_pages, BQ_DEVERR_PAGE);
                    cut = p >= 0;
                } else {
                    cut = p >= 0 || a.s.refs[last] > 1;
                }
            }
        }
        base_s[b] = base;
        want_s[b] = bad ? base : hi;
        mark_s[b] = (p + 1) | (cut ? CUT : 0) | (bad ? BAD : 0);
        last_s[b] = last;
    }
    __syncthreads();
    struct Request {
        int base, want, parent, held, wanted, kept, ask, new_rows;
        bool cut, bad, served;
    };
    auto request = [&](int b) {
        Request r;
        const int mark = mark_s[b];
        r.base = base_s[b], r.want = want_s[b], r.parent = (mark & PARENT) - 1;
        r.cut = mark & CUT, r.bad = mark & BAD, r.served = mark & SERVED;
        r.held = r.bad ? 0 : pages(r.base), r.wanted = r.bad ? 0 : pages(r.want);
        r.kept = r.held - r.cut;  // pages that stay as they are, if it grows
        r.ask = r.wanted > r.kept && r.want > r.base ? r.wanted - r.kept : 0;
        r.new_rows = max(0, r.want - r.base);
        return r;
    };

    // ---- asked pages and rows ----
    const int per = (n + threads - 1) / threads;
    const int b0 = min(n, tid * per), b1 = min(n, b0 + per);
    {
        uint32_t v[2] = {0, 0}, total[2];
        for (int b = b0; b < b1; ++b) {
            const Request r = request(b);
            v[0] = add_up(v[0], r.ask), v[1] = add_up(v[1], r.new_rows);
        }
        scan_threads<2>(v, total, scratch);
        for (int b = b0; b < b1; ++b) {
            const Request r = request(b);
            asked[b] = (int)v[0], rows[b] = (int)v[1];
            v[0] = add_up(v[0], r.ask), v[1] = add_up(v[1], r.new_rows);
        }
        if (tid == 0) asked[n] = (int)total[0], rows[n] = (int)total[1];
    }
    __syncthreads();
    int given = 0, refused = 0;
    for (int b = tid; b < n; b += threads) {
        const Request r = request(b);
        const bool ok = !r.bad && (!r.ask || asked[b + 1] <= count) && (!r.new_rows || rows[b + 1] <= a.t.max_tokens);
        if (ok) mark_s[b] |= SERVED;
        if (ok && r.ask) given = max(given, asked[b + 1]);
        refused += !ok;
    }
    given = __reduce_max_sync(~0u, given);
    refused = __reduce_add_sync(~0u, refused);
    if ((tid & 31) == 0) {
        atomicMax(&s_given, given);
        atomicAdd(&s_refused, refused);
    }
    __syncthreads();
    given = s_given;

    // ---- releases, joined entries and copies of the requests that are served ----
    auto releases = [&](const Request &r) {
        return !r.served || r.parent >= 0 ? 0 : r.cut ? 1 : max(0, r.held - r.wanted);
    };
    auto joins = [&](const Request &r) { return r.served && r.parent >= 0 ? r.kept : 0; };
    int all_joined, all_gone, all_copied;
    {
        uint32_t v[3] = {0, 0, 0}, total[3];
        for (int b = b0; b < b1; ++b) {
            const Request r = request(b);
            v[0] = add_up(v[0], releases(r)), v[1] = add_up(v[1], joins(r)), v[2] += r.served && r.cut;
        }
        scan_threads<3>(v, total, scratch);
        for (int b = b0; b < b1; ++b) {
            const Request r = request(b);
            gone[b] = (int)v[0], joined[b] = (int)v[1], copied[b] = (int)v[2];
            v[0] = add_up(v[0], releases(r)), v[1] = add_up(v[1], joins(r)), v[2] += r.served && r.cut;
        }
        // (a table of 2^31 live entries is larger than any memory: what lies beyond is left alone)
        all_gone = (int)total[0], all_joined = (int)total[1], all_copied = (int)total[2];
        if (tid == 0) gone[n] = all_gone, joined[n] = all_joined, copied[n] = all_copied;
    }
    __syncthreads();
    // every CTA has read lengths, counts, parents' rows and the free count: they may change
    cluster_barrier();

    const int step = (int)cluster * threads, me = (int)rank * threads + tid;
    const int lane = tid & 31;
    auto row_of = [&](int b) { return a.t.table + (long long)b * a.t.table_stride; };
    auto counted = [&](int page) { return page >= 0 && page < pool; };
    // the i-th released page
    auto released = [&](int i) {
        const int b = bq::last_not_above(gone, n, i);
        const Request r = request(b);
        return r.cut ? last_s[b] : row_of(b)[r.wanted + (i - gone[b])];
    };

    // ---- forked rows, counts, popped pages: nothing that one of them writes is read by
    // another, but a parent's last page where the parent takes one of its own ----
    // 32 JOIN entries to a warp at a time, JOIN reads in flight
    constexpr int JOIN = 4;
    for (long long i0 = (long long)(me >> 5) * (32 * JOIN); i0 < all_joined; i0 += (long long)(step >> 5) * (32 * JOIN)) {
        int of[JOIN], col[JOIN], page[JOIN];
        int b = bq::last_not_above(joined, n, (int)min(i0 + lane, (long long)all_joined - 1));
#pragma unroll
        for (int k = 0; k < JOIN; ++k) {
            const long long i = i0 + 32 * k + lane;
            of[k] = -1;
            if (i < all_joined) {
                while (joined[b + 1] <= i) ++b;  // ends: joined[n] > i
                const int p = (mark_s[b] & PARENT) - 1;
                of[k] = b, col[k] = (int)i - joined[b];
                // (the parent may be replacing this entry)
                const bool last = (mark_s[p] & CUT) && col[k] == pages(base_s[p]) - 1;
                page[k] = last ? last_s[p] : row_of(p)[col[k]];
            }
        }
#pragma unroll
        for (int k = 0; k < JOIN; ++k)
            if (of[k] >= 0) {
                row_of(of[k])[col[k]] = page[k];
                if (counted(page[k])) atomicAdd(&a.s.refs[page[k]], 1);
                else atomicOr(&g_status_pages, BQ_DEVERR_PAGE);
            }
    }
    for (long long i = me; i < all_gone; i += step) {
        const int page = released((int)i);
        if (counted(page)) atomicSub(&a.s.refs[page], 1);
        else atomicOr(&g_status_pages, BQ_DEVERR_PAGE);
    }
    for (int i = me; i < given; i += step) {
        const int b = bq::last_not_above(asked, n, i);
        const Request r = request(b);
        const int k = i - asked[b], page = a.t.free_pages[count - 1 - i];
        row_of(b)[r.kept + k] = page;
        if (counted(page)) a.s.refs[page] = 1;
        if (r.cut && k == 0) {
            a.s.copy_src[copied[b]] = last_s[b];
            a.s.copy_dst[copied[b]] = page;
        }
    }
    cluster_barrier();

    // ---- pages that nobody holds any more ----
    long long pushed = 0;
    if (all_gone) {
        for (long long i = me; i < all_gone; i += step) {
            const int page = released((int)i);
            if (counted(page) && __ldcg(&a.s.refs[page]) <= 0) atomicMin(&a.s.refs[page], CLAIM + (int)i);
        }
        cluster_barrier();
        // each thread a run of releases
        const long long run = ((long long)all_gone + step - 1) / step;
        const long long i0 = min((long long)all_gone, me * run), i1 = min((long long)all_gone, i0 + run);
        auto mine = [&](long long i, int &page) {
            page = released((int)i);
            return counted(page) && __ldcg(&a.s.refs[page]) == CLAIM + (int)i;
        };
        uint32_t v[1] = {0}, total[1];
        for (long long i = i0; i < i1; ++i) {
            int page;
            v[0] += mine(i, page);
        }
        scan_threads<1>(v, total, scratch);
        if (tid == 0) s_pushed = total[0];
        cluster_barrier();
        long long before = 0;
        for (uint32_t k = 0; k < cluster; ++k) {
            const long long p = peer_word(&s_pushed, k);
            before += k < rank ? p : 0;
            pushed += p;
        }
        long long at = count - given + before + v[0];
        for (long long i = i0; i < i1; ++i) {
            int page;
            if (!mine(i, page)) continue;
            a.s.refs[page] = 0;
            if (at < pool) a.t.free_pages[at] = page;
            ++at;
        }
    }

    // ---- outputs ----
    if (with_rows) {
        const long long all = min((long long)rows[n], (long long)a.t.max_tokens);
        for (long long t = me; t < a.t.max_tokens; t += step) {
            long long slot = -1;
            int position = 0;
            if (t < all) {
                const int b = bq::last_not_above(rows, n, (int)t);
                if (mark_s[b] & SERVED) {
                    position = base_s[b] + (int)(t - rows[b]);
                    const int q = (int)a.page.div((uint32_t)position);
                    slot = (long long)__ldcg(row_of(b) + q) * a.t.page_size + (position - q * a.t.page_size);
                }
            }
            a.t.slots[t] = slot;
            a.t.positions[t] = position;
        }
    }
    for (int b = me; b <= n; b += step) a.t.starts[b] = rows[b];
    for (int b = me; b < n; b += step) {
        const int mark = mark_s[b];
        // a refused fork stays empty
        a.t.lens_out[b] = mark & SERVED ? want_s[b] : (mark & PARENT) ? 0 : base_s[b];
        if (b >= all_copied) a.s.copy_src[b] = a.s.copy_dst[b] = -1;
    }
    if (me == 0) {
        const long long left = count - given + pushed;
        if (left > pool) atomicOr(&g_status_pages, BQ_DEVERR_POOL);
        *a.t.free_count_out = (int)min(left, (long long)pool);
        *a.t.refused = s_refused;
        *a.s.copy_count = all_copied;
    }
    cluster_barrier();  // shared memory stays until the others have read it
}

// ---------------------------------------------------------------------------
// compaction
// ---------------------------------------------------------------------------
struct CompactArgs {
    bq_kv_compact_args c;
    bq::FastDiv page;
};

__global__ void __launch_bounds__(THREADS) compact_kernel(const __grid_constant__ CompactArgs a) {
    __shared__ uint32_t scratch[1][WARPS];
    constexpr int KEPT = 64;
    __shared__ uint32_t words[WARPS][KEPT];
    __shared__ long long s_live, s_moves;  // pages in use in this CTA's part; moves, in the CTA that meets them
    bq::pdl_wait();
    bq::pdl_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_rank(), cluster = cluster_size();
    const long long pool = a.c.pool;
    const int *refs = a.c.refs;
    // a run of pages for each warp
    const long long warps = (long long)cluster * WARPS;
    const long long run = (pool + warps * 32 - 1) / (warps * 32) * 32;
    const long long p0 = min(pool, (rank * WARPS + warp) * run), p1 = min(pool, p0 + run);
    // which of its pages are in use, a word for 32 of them, if there is room for all
    const bool kept = run <= 32 * KEPT;
    constexpr int READS = 8;  // in flight
    auto look = [&](long long q0, auto tell) {  // the run's words from page q0 on, READS of them
        bool live[READS];
#pragma unroll
        for (int k = 0; k < READS; ++k) {
            const long long p = q0 + 32 * k + lane;
            live[k] = p < p1 && refs[p] > 0;
        }
#pragma unroll
        for (int k = 0; k < READS; ++k) tell(k, __ballot_sync(~0u, live[k]));
    };
    uint32_t v[1] = {0}, total[1];
    for (long long q0 = p0; q0 < p1; q0 += 32 * READS)
        look(q0, [&](int k, uint32_t bits) {
            if (lane == 0) {
                v[0] += __popc(bits);
                const long long at = (q0 - p0) / 32 + k;
                if (kept && at < KEPT) words[warp][at] = bits;
            }
        });
    __syncwarp();
    scan_threads<1>(v, total, scratch);  // pages in use before each warp's, from its first thread
    long long before = __shfl_sync(~0u, v[0], 0);  // right for lane 0
    if (tid == 0) s_live = total[0], s_moves = -1;
    cluster_barrier();
    long long many = 0;  // pages in use
    for (uint32_t k = 0; k < cluster; ++k) {
        const long long n = peer_word(&s_live, k);
        before += k < rank ? n : 0;
        many += n;
    }
    // moves: the pages below `many` that are free, as many as the ones in use from there on
    if (p0 <= many && many < p1) {
        long long live = 0;
        for (long long p = p0 + lane; p < many; p += 32) live += refs[p] > 0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) live += __shfl_xor_sync(~0u, live, o);
        if (lane == 0) s_moves = many - (before + live);
    }
    cluster_barrier();
    long long moves = 0;
    for (uint32_t k = 0; k < cluster; ++k) moves = max(moves, peer_word(&s_moves, k));
    const long long room = a.c.max_moves, done = min(moves, room);
    auto place = [&](long long q0, uint32_t bits) {  // 32 pages
        const long long p = q0 + lane;
        const bool in = p < p1, live = bits >> lane & 1;
        const long long below = before + __popc(bits & ((1u << lane) - 1));  // pages in use below p
        before += __popc(bits);
        if (!in) return;
        a.c.moved[p] = (int)p;
        const long long above = many - below - live;  // pages in use above p
        if (p >= many) {
            if (live && above < done) a.c.copy_src[above] = (int)p;
            if (!live || above < done)
                a.c.free_pages[pool - 1 - p - max(0LL, above - done)] = (int)p;
        } else if (!live) {
            const long long rank_of = p - below;  // among the free pages
            if (rank_of < done) a.c.copy_dst[rank_of] = (int)p;
            else a.c.free_pages[pool - many - (moves - done) + moves - 1 - rank_of] = (int)p;
        }
    };
    if (kept) {
        for (long long q0 = p0; q0 < p1; q0 += 32) place(q0, words[warp][(q0 - p0) / 32]);
    } else {
        for (long long q0 = p0; q0 < p1; q0 += 32 * READS)
            look(q0, [&](int k, uint32_t bits) { place(q0 + 32 * k, bits); });
    }
    for (long long i = done + rank * THREADS + tid; i < room; i += (long long)cluster * THREADS)
        a.c.copy_src[i] = a.c.copy_dst[i] = -1;
    if (rank == 0 && tid == 0) {
        *a.c.copy_count = (int)done;
        *a.c.free_count_out = (int)(pool - many);
    }
    cluster_barrier();  // everyone has read the counts, and the lists are complete
    for (long long i = rank * THREADS + tid; i < done; i += (long long)cluster * THREADS) {
        const int from = __ldcg(a.c.copy_src + i), to = __ldcg(a.c.copy_dst + i);
        a.c.refs[to] = __ldcg(refs + from);
        a.c.refs[from] = 0;
        a.c.moved[from] = to;
    }
}

// the tables' entries by their pages' new numbers
constexpr int RENUMBER_THREADS = 256;
__global__ void __launch_bounds__(RENUMBER_THREADS) renumber_kernel(const __grid_constant__ CompactArgs a) {
    bq::pdl_wait();
    const int b = blockIdx.y;
    const long long most = (long long)a.c.table_width * a.c.page_size;
    const int len = (int)min((long long)max(a.c.lens[b], 0), most);
    const uint32_t q = a.page.div((uint32_t)len);
    const int held = (int)(q + ((uint32_t)len - q * a.page.d != 0));
    int *row = a.c.table + (long long)b * a.c.table_stride;
    for (int c = blockIdx.x * RENUMBER_THREADS + threadIdx.x; c < held; c += gridDim.x * RENUMBER_THREADS) {
        const int page = row[c];
        if (page >= 0 && page < a.c.pool) {
            const int now = a.c.moved[page];
            if (now != page) row[c] = now;
        } else {
            atomicOr(&g_status_pages, BQ_DEVERR_PAGE);
        }
    }
}

// ---------------------------------------------------------------------------
// copies
// ---------------------------------------------------------------------------
constexpr int COPY_THREADS = 256, COPY_EACH = 4, COPY_CACHES = 96;

// one plane of a page as runs of contiguous bytes: n2 x n1 of them
struct Plane {
    uint32_t vec;      // bytes of an access
    bq::FastDiv run;   // accesses of a run
    bq::FastDiv n1;
    uint32_t all;      // accesses of a page
    uint32_t pieces;   // CTA turns of a page
    long long page, s1, s2;  // bytes from page to page and run to run
};
struct CopyArgs {
    Plane data, scales;
    int caches, kinds;  // kinds: 2 planes, or 4 with scales
    long long pairs, pages;
    uint32_t units;     // of a pair
    bq::FastDiv per_cache;
    const int *src, *dst, *count;
    void *plane[COPY_CACHES][4];
};

template <class V>
__device__ __forceinline__ void copy_piece(const Plane &p, uint8_t *base, long long from, long long to, uint32_t piece) {
    V v[COPY_EACH];
    long long at[COPY_EACH];
#pragma unroll
    for (int k = 0; k < COPY_EACH; ++k) {
        const uint32_t i = piece * (COPY_THREADS * COPY_EACH) + k * COPY_THREADS + threadIdx.x;
        at[k] = -1;
        if (i < p.all) {
            const uint32_t r = p.run.div(i), r2 = p.n1.div(r);
            at[k] = (long long)r2 * p.s2 + (long long)(r - r2 * p.n1.d) * p.s1 + (long long)(i - r * p.run.d) * (int)sizeof(V);
            v[k] = *reinterpret_cast<const V *>(base + from * p.page + at[k]);
        }
    }
#pragma unroll
    for (int k = 0; k < COPY_EACH; ++k)
        if (at[k] >= 0) *reinterpret_cast<V *>(base + to * p.page + at[k]) = v[k];
}

__global__ void __launch_bounds__(COPY_THREADS) copy_kernel(const __grid_constant__ CopyArgs a) {
    bq::pdl_wait();
    const long long pairs = a.count ? min(a.pairs, (long long)max(*a.count, 0)) : a.pairs;
    const long long units = pairs * a.units;
    for (long long u = blockIdx.x; u < units; u += gridDim.x) {
        const long long pair = u / a.units;
        const int from = a.src[pair], to = a.dst[pair];
        if (from < 0 || to < 0 || from == to) continue;
        if (from >= a.pages || to >= a.pages) {
            if (threadIdx.x == 0) atomicOr(&g_status_pages, BQ_DEVERR_PAGE);
            continue;
        }
        const uint32_t rest = (uint32_t)(u - pair * a.units);
        const uint32_t cache = a.per_cache.div(rest);
        uint32_t piece = rest - cache * a.per_cache.d;
        const bool scales = piece >= 2 * a.data.pieces;
        if (scales) piece -= 2 * a.data.pieces;
        const uint32_t each = scales ? a.scales.pieces : a.data.pieces;
        const uint32_t second = piece >= each;
        if (second) piece -= each;
        uint8_t *base = static_cast<uint8_t *>(a.plane[cache][(scales ? 2 : 0) + second]);
        if (!scales) {
            copy_piece<uint4>(a.data, base, from, to, piece);
        } else if (a.scales.vec == 16) {
            copy_piece<uint4>(a.scales, base, from, to, piece);
        } else if (a.scales.vec == 8) {
            copy_piece<uint2>(a.scales, base, from, to, piece);
        } else {
            copy_piece<uint16_t>(a.scales, base, from, to, piece);
        }
    }
}

// a plane whose elements are `bytes` wide and `per` values of the cache each
Plane plane_of(const bq_kv_cache &c, int bytes, int per, int widest) {
    const long long D = c.head_dim / per, H = c.kv_heads, S = c.page_size;
    const long long hs = H > 1 ? c.head_stride / per : 0, ss = S > 1 ? c.slot_stride / per : 0;
    long long run = D, n1 = 1, n2 = 1, s1 = 0, s2 = 0;
    // (a dimension of one entry has no stride)
    if (S == 1 || ss == D) {  // a head's slots are a run
        run = S * D;
        if (H == 1 || hs == run) run *= H;
        else n1 = H, s1 = hs;
    } else if (H == 1 || hs == D) {  // a slot's heads are
        run = H * D;
        if (ss == run) run *= S;
        else n1 = S, s1 = ss;
    } else {
        n1 = S, s1 = ss, n2 = H, s2 = hs;
    }
    Plane p;
    p.page = c.pages > 1 ? c.page_stride / per * bytes : 0;
    p.s1 = s1 * bytes, p.s2 = s2 * bytes;
    p.vec = (uint32_t)widest;
    while (p.vec > (uint32_t)bytes && (run * bytes % p.vec || p.s1 % p.vec || p.s2 % p.vec || p.page % p.vec)) p.vec /= 2;
    if (p.vec == 4) p.vec = 2;  // (16, 8 and 2 byte accesses)
    p.run.set((uint32_t)(run * bytes / p.vec));
    p.n1.set((uint32_t)n1);
    p.all = (uint32_t)(run * bytes / p.vec * n1 * n2);
    p.pieces = (p.all + COPY_THREADS * COPY_EACH - 1) / (COPY_THREADS * COPY_EACH);
    return p;
}

// CTAs of a cluster for much work: 16 where the device takes such a cluster with
// this much shared memory (the atomics of a step's forks and the reads of a large
// pool are shared out among twice the SMs), else 8
template <class K>
int largest_cluster(K *kern, size_t smem) {
    static std::atomic<int> known[64];  // per device: 0 not asked yet
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return CLUSTER;
    int n = known[dev].load();
    if (n) return n;
    n = CLUSTER;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(CLUSTER_MOST);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = CLUSTER_MOST, attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int fit = 0;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
        cudaOccupancyMaxActiveClusters(&fit, kern, &cfg) == cudaSuccess && fit > 0)
        n = CLUSTER_MOST;
    cudaGetLastError();
    known[dev].store(n);
    return n;
}

}  // namespace

int bq_internal_status_pages(unsigned int *flags, int clear) { return read_status_pages(flags, clear); }

extern "C" bq_status bq_kv_shared_tables(const bq_kv_tables *t, const bq_kv_sharing *s, void *stream) {
    if (!s) return BQ_ERR_NULL;
    const bq_status st = bq::check_tables(t);
    if (st != BQ_OK) return st;
    if (!s->refs || !s->copy_count || (t->requests && (!s->copy_src || !s->copy_dst))) return BQ_ERR_NULL;
    const void *words[] = {s->parents, s->refs, s->copy_src, s->copy_dst, s->copy_count};
    for (const void *p : words)
        if (!bq::aligned_to(p, 4)) return BQ_ERR_ALIGN;
    ShareArgs a;
    a.t = *t;
    a.s = *s;
    a.page.set((uint32_t)t->page_size);
    const bool with_rows = t->max_tokens <= bq::TABLES_ROWS_ALONE;
    // one CTA for a step that cannot move much, however it turns out
    const long long work = (with_rows ? t->max_tokens : 0) + (long long)t->requests * t->table_width;
    const size_t smem = (size_t)(9 * t->requests + 5) * sizeof(int);
    constexpr int SMEM_MOST = (int)((9 * bq::TABLES_MAX_REQUESTS + 5) * sizeof(int));
    if (smem > 40 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(share_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_MOST);
        if (e != cudaSuccess) return bq::from_cuda_error(e);
    }
    // (asked with what every call of up to 1000 requests needs; more take 8 CTAs)
    const int cluster = work <= 16LL * THREADS                ? 1
                        : work <= 256LL * THREADS || smem > 40 * 1024 ? CLUSTER
                                                              : largest_cluster(share_kernel, 40 * 1024);
    // (a barrier of 32 warps costs more than the work of a small step)
    const int threads = cluster == 1 && t->requests <= 256 ? 256 : THREADS;
    const cudaError_t e = bq::launch_pdl(share_kernel, dim3((unsigned)cluster), threads, smem, stream, cluster, a,
                                         (int)with_rows);
    if (e != cudaSuccess || with_rows) return bq::from_cuda_error(e);
    return bq::from_cuda_error(bq::rows_launch(a.t, stream));
}

extern "C" bq_status bq_kv_compact(const bq_kv_compact_args *c, void *stream) {
    if (!c) return BQ_ERR_NULL;
    if (c->requests < 0 || c->requests > bq::TABLES_MAX_REQUESTS || c->page_size < 1 || c->page_size > 65536 ||
        c->table_width < 1 || c->table_stride < c->table_width || c->table_stride > (1LL << 40) || c->pool < 1 ||
        c->pool == 0x7fffffff || c->max_moves < 0 || c->max_moves > 0x7ffffffeLL)
        return BQ_ERR_SHAPE;
    if (!c->free_pages || !c->refs || !c->copy_count || !c->moved || !c->free_count_out) return BQ_ERR_NULL;
    if (c->requests && (!c->lens || !c->table)) return BQ_ERR_NULL;
    if (c->max_moves && (!c->copy_src || !c->copy_dst)) return BQ_ERR_NULL;
    const void *words[] = {c->lens, c->table, c->free_pages, c->refs, c->copy_src, c->copy_dst, c->copy_count,
                           c->moved, c->free_count_out};
    for (const void *p : words)
        if (!bq::aligned_to(p, 4)) return BQ_ERR_ALIGN;
    CompactArgs a;
    a.c = *c;
    a.page.set((uint32_t)c->page_size);
    const int cluster = c->pool <= 4 * THREADS ? 1 : c->pool <= 32 * THREADS ? CLUSTER : largest_cluster(compact_kernel, 0);
    cudaError_t e = bq::launch_pdl(compact_kernel, dim3((unsigned)cluster), THREADS, 0, stream, cluster, a);
    if (e != cudaSuccess || c->requests == 0) return bq::from_cuda_error(e);
    const int across = (c->table_width + RENUMBER_THREADS * 4 - 1) / (RENUMBER_THREADS * 4);
    e = bq::launch_pdl(renumber_kernel, dim3((unsigned)across, (unsigned)c->requests), RENUMBER_THREADS, 0, stream, 1, a);
    return bq::from_cuda_error(e);
}

extern "C" bq_status bq_kv_copy_pages(const bq_kv_cache *const *caches, int n, const int32_t *src, const int32_t *dst,
                                      const int32_t *count, int64_t pairs, void *stream) {
    if (n < 0 || pairs < 0 || pairs > 0x7fffffffLL) return BQ_ERR_SHAPE;
    if (n == 0) return BQ_OK;
    if (!caches || !caches[0]) return BQ_ERR_NULL;
    const bq_kv_cache &c = *caches[0];
    for (int i = 0; i < n; ++i) {
        if (!caches[i]) return BQ_ERR_NULL;
        const bq_kv_cache &o = *caches[i];
        const bq_status s = bq::check_cache_shape(&o);
        if (s != BQ_OK) return s;
        if (o.type != c.type || o.kv_heads != c.kv_heads || o.head_dim != c.head_dim || o.page_size != c.page_size ||
            o.pages != c.pages || o.page_stride != c.page_stride || o.head_stride != c.head_stride ||
            o.slot_stride != c.slot_stride)
            return BQ_ERR_SHAPE;
    }
    // accesses of a page are counted in 32 bits
    if ((int64_t)c.kv_heads * c.page_size * c.head_dim > (1LL << 30)) return BQ_ERR_SHAPE;
    if (pairs == 0) return BQ_OK;
    for (int i = 0; i < n; ++i) {
        const bq_status s = bq::check_cache_pointers(caches[i]);
        if (s != BQ_OK) return s;
    }
    if (!src || !dst) return BQ_ERR_NULL;
    if (!bq::aligned_to(src, 4) || !bq::aligned_to(dst, 4) || !bq::aligned_to(count, 4)) return BQ_ERR_ALIGN;
    const int sms = bq::device_sms();
    if (!sms) return BQ_ERR_CUDA;
    CopyArgs a;
    const bool q8 = c.type == BQ_Q8_0;
    a.kinds = q8 ? 4 : 2;
    a.data = plane_of(c, q8 ? 1 : 2, 1, 16);
    int widest = 16;  // of the scales: their planes start on 8 bytes
    for (int i = 0; i < n && q8; ++i)
        if (!bq::aligned_to(caches[i]->k_scale, 16) || !bq::aligned_to(caches[i]->v_scale, 16)) widest = 8;
    a.scales = plane_of(c, 2, 32, widest);
    const uint32_t per = 2 * (a.data.pieces + (q8 ? a.scales.pieces : 0));
    a.per_cache.set(per);
    a.pairs = pairs, a.pages = c.pages;
    a.src = src, a.dst = dst, a.count = count;
    for (int i0 = 0; i0 < n; i0 += COPY_CACHES) {
        a.caches = n - i0 < COPY_CACHES ? n - i0 : COPY_CACHES;
        for (int i = 0; i < a.caches; ++i) {
            const bq_kv_cache &o = *caches[i0 + i];
            a.plane[i][0] = o.k, a.plane[i][1] = o.v;
            a.plane[i][2] = o.k_scale, a.plane[i][3] = o.v_scale;
        }
        if ((uint64_t)per * a.caches > 0x7fffffffull) return BQ_ERR_SHAPE;
        a.units = per * (uint32_t)a.caches;
        const int64_t all = pairs * a.units, most = (int64_t)sms * 8;
        const cudaError_t e = bq::launch_pdl(copy_kernel, dim3((unsigned)(all < most ? all : most)), COPY_THREADS, 0, stream,
                                             1, a);
        if (e != cudaSuccess) return bq::from_cuda_error(e);
    }
    return BQ_OK;
}
