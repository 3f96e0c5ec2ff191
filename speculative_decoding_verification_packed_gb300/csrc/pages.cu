// pages.cu -- the pages of a cache: giving them to requests and taking them back, sharing them between
// requests, and moving them together.
//
// What is decided (which free page goes where) depends on everything before it in order, so one cluster
// of eight blocks decides it: counts are exchanged through distributed shared memory, and a cluster
// barrier stands between what one phase writes and the next reads.  A single block would read a pool of
// 262144 pages' counts alone; a grid would need a launch for each phase.  What is only work, copies of
// pages and of table rows, is a second kernel over all SMs, a dependent of the first.
//
// Free pages are found by their counts (refs == 0), lowest ids first: no list of free pages has to be
// kept consistent, and the ids in use stay low.  A warp looks at 32 pages a load; ballots rank them.
//
// What bounds it: for a step's few pages the chain of dependent reads and cluster barriers (64 requests: 8.2 us of a
// graph's 9.7); for 54700 pages given back at once their atomics (12 of 21 us); for moves memory (924 MB in a compaction:
// 150 us, 6.2 TB/s).
#include <cstring>

#include "svp_cache.cuh"

namespace svp {

constexpr int kPgCluster = 8, kPgThreads = 1024, kPgWarps = kPgThreads / 32;
constexpr int kPgMost = 8;            // units of 32 pages that a warp has in one window, at most
constexpr int kPgRequests = 1024;     // requests, or forks, of a call: one a thread

struct PagesParams {
    int32_t *table, *used, *refs;
    int32_t n, max_pages, page_shift, num_pages;
    const int32_t *src, *dst, *length;
    int32_t forks;
    int32_t *live;
    int32_t *status;
    int4 *plan;                       // fork: (source, destination, whole pages or -1, page of the part or -1)
    int32_t *tail;                    // fork: page of the part
    int32_t *holes, *movers, *rank;   // compact: the moves' ends, and of a page its place among the movers
    int32_t *moves;                   // their number, and L
};

struct PagesCaches {
    void *k[SVP_PAGES_MAX_CACHES], *v[SVP_PAGES_MAX_CACHES];
    uint8_t *k_exp[SVP_PAGES_MAX_CACHES], *v_exp[SVP_PAGES_MAX_CACHES];
    int64_t s_page, s_head, s_tok;    // bytes
    int32_t count, hkv, row_shift;    // 2^row_shift 16-byte pieces in a (token, head) row
};

// ------------------------------------------------------------------ cluster
__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// Barrier of every thread of the cluster.  What a thread that says `wrote` has written before it is seen by all after
// it; warps without such a thread pay no fence (a window's 0.3 us otherwise).
__device__ __forceinline__ void cluster_sync(bool wrote)
{
    if (__any_sync(0xffffffffu, wrote))
        asm volatile("fence.acq_rel.cluster;" ::: "memory");
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ uint64_t cluster_load64(const uint64_t *x, uint32_t rank)   // block rank's copy of x
{
    uint64_t v;
    asm volatile("{\n\t.reg .b32 a;\n\t"
                 "mapa.shared::cluster.u32 a, %1, %2;\n\t"
                 "ld.shared::cluster.b64 %0, [a];\n\t}"
                 : "=l"(v)
                 : "r"(smem_u32(x)), "r"(rank)
                 : "memory");
    return v;
}

__device__ __forceinline__ int32_t cluster_load(const int32_t *x, uint32_t rank)
{
    int32_t v;
    asm volatile("{\n\t.reg .b32 a;\n\t"
                 "mapa.shared::cluster.u32 a, %1, %2;\n\t"
                 "ld.shared::cluster.s32 %0, [a];\n\t}"
                 : "=r"(v)
                 : "r"(smem_u32(x)), "r"(rank)
                 : "memory");
    return v;
}

struct PagesShared {
    uint64_t both[kPgWarps];
    uint64_t units[2][kPgWarps], sum[2][2];   // counts of a window's units, 16 bits each: of the warps; of this block,
                                              // of even and odd windows
    int32_t warp[kPgWarps];
    int32_t tot[2];
    int32_t need[kPgRequests + 1], drop[kPgRequests + 1];   // before each request
    int32_t a[kPgRequests], b[kPgRequests];
};

// Exclusive prefix sums of need and drop (both below 2^31 in all) over the block's threads into s.need and s.drop
// [0 .. kPgThreads]; ends in a barrier.
__device__ __forceinline__ void pages_scan(PagesShared &s, int32_t need, int32_t drop)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint64_t incl = (uint64_t)(uint32_t)need | (uint64_t)(uint32_t)drop << 32;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o)
            incl += v;
    }
    if (lane == 31)
        s.both[warp] = incl;
    __syncthreads();
    uint64_t w = s.both[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t v = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o)
            w += v;
    }
    const uint64_t ahead = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
    incl += warp == 0 ? 0 : ahead;
    s.need[threadIdx.x + 1] = (int32_t)incl;
    s.drop[threadIdx.x + 1] = (int32_t)(incl >> 32);
    if (threadIdx.x == 0)
        s.need[0] = s.drop[0] = 0;
    __syncthreads();
}

__device__ __forceinline__ int32_t pages_owner(const int32_t *before, int32_t n, int32_t x)   // before[i] <= x < before[i + 1]
{
    int32_t lo = 0, hi = n;
    while (hi - lo > 1) {
        const int32_t mid = (lo + hi) >> 1;
        if (before[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// The cluster's sum of `mine` (one value a block, in every thread), and that of the blocks before this one.
// Uses s.tot[w & 1], which calls with the other w leave alone.
__device__ __forceinline__ int32_t pages_total(PagesShared &s, uint32_t rank, uint32_t w, int32_t mine, int32_t &before)
{
    if (threadIdx.x == 0)
        s.tot[w & 1] = mine;
    cluster_sync(threadIdx.x == 0);
    const int lane = threadIdx.x & 31;
    int32_t v = lane < kPgCluster ? cluster_load(&s.tot[w & 1], lane) : 0;
#pragma unroll
    for (int o = 1; o < kPgCluster; o <<= 1) {
        const int32_t u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o && lane < kPgCluster)
            v += u;
    }
    before = rank == 0 ? 0 : __shfl_sync(0xffffffffu, v, (int)(rank + 31) & 31);
    return __shfl_sync(0xffffffffu, v, kPgCluster - 1);
}

// Calls take(r, page) for the free pages with ranks r < need, by id; returns how many were looked up, which is
// less than need only if there are no more.  A window is `each` units of 32 pages a warp, dealt out in turn, so that the
// first free pages, which are the ones that are taken, are spread over all blocks.
template <class F>
__device__ __forceinline__ int32_t pages_find(const PagesParams &p, PagesShared &s, uint32_t rank, int32_t need, F take)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t spread = ((int64_t)p.num_pages + kPgCluster * kPgThreads - 1) / (kPgCluster * kPgThreads);
    const int each = (int)(spread < kPgMost ? spread : kPgMost);
    int32_t found = 0;
    uint32_t w = 0;
    for (int64_t base = 0; base < p.num_pages && found < need; base += (int64_t)each * kPgCluster * kPgThreads, ++w) {
        const int64_t first = base + ((int64_t)rank * kPgWarps + warp) * 32 + lane;
        uint32_t mask[kPgMost];
        uint64_t cnt[2] = {0, 0};                         // (a unit's counts are at most 8192 over the cluster)
#pragma unroll
        for (int u = 0; u < kPgMost; ++u) {
            const int64_t page = first + u * (kPgCluster * kPgThreads);
            mask[u] = __ballot_sync(0xffffffffu, u < each && page < p.num_pages && __ldcg(p.refs + page) == 0);
            cnt[u >> 2] |= (uint64_t)__popc(mask[u]) << (16 * (u & 3));
        }
        if (lane < 2)
            s.units[lane][warp] = cnt[lane];
        __syncthreads();
        uint64_t at[2], all[2];                           // free pages of each unit before this warp's, and in all
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            at[x] = all[x] = 0;
            if (x * 4 >= each)
                continue;
            uint64_t v = s.units[x][lane];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint64_t y = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o)
                    v += y;
            }
            const uint64_t ahead = __shfl_sync(0xffffffffu, v, (warp + 31) & 31);
            at[x] = warp == 0 ? 0 : ahead;
            if (threadIdx.x == kPgThreads - 1)
                s.sum[w & 1][x] = v;                      // (the other pair is still read, in the window before)
        }
        cluster_sync(threadIdx.x == kPgThreads - 1);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            if (x * 4 >= each)
                continue;
            uint64_t v = lane < kPgCluster ? cluster_load64(&s.sum[w & 1][x], lane) : 0;
#pragma unroll
            for (int o = 1; o < kPgCluster; o <<= 1) {
                const uint64_t y = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o && lane < kPgCluster)
                    v += y;
            }
            const uint64_t ahead = __shfl_sync(0xffffffffu, v, (int)(rank + 31) & 31);
            at[x] += rank == 0 ? 0 : ahead;
            all[x] = __shfl_sync(0xffffffffu, v, kPgCluster - 1);
        }
#pragma unroll
        for (int u = 0; u < kPgMost; ++u) {
            const int32_t r = found + (int32_t)(at[u >> 2] >> (16 * (u & 3)) & 0xffffu) + __popc(mask[u] & ((1u << lane) - 1u));
            if ((mask[u] >> lane & 1u) && r < need)
                take(r, (int32_t)(first + u * (kPgCluster * kPgThreads)));
            found += (int32_t)(all[u >> 2] >> (16 * (u & 3)) & 0xffffu);
        }
    }
    return found;
}

// ------------------------------------------------------------------ resize
__global__ void __cluster_dims__(kPgCluster, 1, 1) __launch_bounds__(kPgThreads)
    pages_resize_kernel(const __grid_constant__ PagesParams p)
{
    __shared__ PagesShared s;
    griddep_launch_dependents();
    griddep_wait();
    const uint32_t rank = cluster_rank();
    const int32_t i = threadIdx.x;
    // Block 0 looks at the requests, the others take its numbers: all agree on them (and on the number of
    // barriers) whatever else changes the tables meanwhile.  Block 1 looks at them for the last pages of those that keep
    // their number of pages, which tells no more than a status bit and would lengthen block 0's chain of reads.
    int32_t held = 0, want = 0, bits = 0;
    if (rank <= 1 && i < p.n) {
        const int32_t len = __ldg(p.length + i);
        held = __ldcg(p.used + i);
        want = held;
        if (held < 0 || held > p.max_pages) {
            bits = SVP_DEV_BAD_CONTEXT;
            held = want = 0;
        } else if (len >= 0) {
            const int32_t part = len & ((1 << p.page_shift) - 1);
            want = (len >> p.page_shift) + (part ? 1 : 0);
            if (want > p.max_pages) {
                bits = SVP_DEV_BAD_CONTEXT;
                want = held;
            } else if (part && (rank == 0 ? want < held : want == held)) {
                // the last page is kept in part: it has to be this request's alone
                const int32_t page = __ldcg(p.table + (int64_t)i * p.max_pages + want - 1);
                if (page >= 0 && page < p.num_pages && __ldcg(p.refs + page) > 1) {
                    bits = SVP_DEV_BAD_CONTEXT;
                    want = held;
                }
            }
        }
    }
    if (rank == 0) {
        s.a[i] = held;
        s.b[i] = want;
        // (sums of up to 1024 x max_pages < 2^31: checked on the host)
        pages_scan(s, max(want - held, 0), max(held - want, 0));
    }
    cluster_sync(rank <= 1);
    if (rank != 0) {
        // (of the requests that there are: block 0 answers for seven)
        if (i < p.n) {
            s.a[i] = cluster_load(&s.a[i], 0);
            s.b[i] = cluster_load(&s.b[i], 0);
            s.need[i + 1] = cluster_load(&s.need[i + 1], 0);
            s.drop[i + 1] = cluster_load(&s.drop[i + 1], 0);
        }
        if (i == 0)
            s.need[0] = s.drop[0] = 0;
        __syncthreads();
    }
    const int32_t need = s.need[p.n], drop = s.drop[p.n];
    if (drop > 0) {
        // (four entries a thread in flight; 54700 entries take 12 us of a call's 21, bound by their blocks' atomics)
        constexpr int U = 4, kAll = kPgCluster * kPgThreads;
        for (int32_t x0 = (int32_t)rank * kPgThreads + i; x0 < drop; x0 += U * kAll) {
            int32_t page[U], old[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t x = x0 + (int64_t)u * kAll;
                page[u] = -1;
                if (x < drop) {
                    const int32_t q = pages_owner(s.drop, p.n, (int32_t)x);
                    int32_t *at = p.table + (int64_t)q * p.max_pages + s.b[q] + ((int32_t)x - s.drop[q]);
                    page[u] = __ldcg(at);
                    *at = -1;
                    if (page[u] < 0 || page[u] >= p.num_pages) {
                        page[u] = -1;
                        bits |= SVP_DEV_BAD_CONTEXT;
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                old[u] = page[u] >= 0 ? atomicSub(p.refs + page[u], 1) : 1;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (old[u] <= 0) {                        // (a count that was none already)
                    atomicAdd(p.refs + page[u], 1);
                    bits |= SVP_DEV_BAD_CONTEXT;
                }
            }
            if (drop - x0 <= U * kAll)
                break;                                    // (x0 may not pass 2^31)
        }
        cluster_sync((int32_t)rank * kPgThreads + i < drop);
    }
    int32_t found = 0;
    if (need > 0) {
        found = pages_find(p, s, rank, need, [&](int32_t r, int32_t page) {
            const int32_t q = pages_owner(s.need, p.n, r);
            p.table[(int64_t)q * p.max_pages + s.a[q] + (r - s.need[q])] = page;
            p.refs[page] = 1;
        });
        if (found < need) {
            // the request that the last pages did not suffice for gives its own back
            cluster_sync(true);
            const int32_t q = pages_owner(s.need, p.n, found);
            for (int32_t x = s.need[q] + i; rank == 0 && x < found; x += kPgThreads) {
                int32_t *at = p.table + (int64_t)q * p.max_pages + s.a[q] + (x - s.need[q]);
                p.refs[__ldcg(at)] = 0;
                *at = -1;
            }
            if (rank == 0 && i == 0)
                bits |= SVP_DEV_NO_PAGES;
        }
    }
    if (rank == 0 && i < p.n && want != held && (want < held || s.need[i + 1] <= found))
        p.used[i] = want;
    if (bits)
        set_status(p.status, bits);
    cluster_sync(false);                                       // (no block leaves while another reads its counts)
}

// ------------------------------------------------------------------ fork
__global__ void __cluster_dims__(kPgCluster, 1, 1) __launch_bounds__(kPgThreads)
    pages_fork_kernel(const __grid_constant__ PagesParams p)
{
    __shared__ PagesShared s;
    griddep_launch_dependents();
    griddep_wait();
    const uint32_t rank = cluster_rank();
    const int32_t f = threadIdx.x;
    s.a[f] = INT32_MAX;                                   // by request: the first fork into it
    __syncthreads();
    int32_t from = 0, to = 0, whole = -1, part = 0, bits = 0;
    bool fine = false, lost = false;                      // lost: the part's page is none of the pool
    if (rank == 0 && f < p.forks) {                       // (as in the resize)
        from = __ldg(p.src + f);
        to = __ldg(p.dst + f);
        const int32_t len = __ldg(p.length + f);
        if (from < 0 || from >= p.n || to < 0 || to >= p.n) {
            bits = SVP_DEV_BAD_SLOTS;
        } else {
            // (the entry beside the counts: one round trip)
            const bool row = len >= 0 && (len >> p.page_shift) < p.max_pages;
            const int32_t page = row ? __ldcg(p.table + (int64_t)from * p.max_pages + (len >> p.page_shift)) : -1;
            const int32_t held = __ldcg(p.used + from);
            if (__ldcg(p.used + to) != 0) {
                bits = SVP_DEV_BAD_SLOTS;
            } else if (len < 0 || held < 0 || held > p.max_pages || len > ((int64_t)held << p.page_shift)) {
                bits = SVP_DEV_BAD_CONTEXT;
            } else {
                fine = true;
                whole = len >> p.page_shift;
                part = len & ((1 << p.page_shift) - 1);
                lost = part && (page < 0 || page >= p.num_pages);
                atomicMin(&s.a[to], f);
            }
        }
    }
    __syncthreads();
    if (fine && s.a[to] != f) {
        fine = false;
        bits = SVP_DEV_BAD_SLOTS;
    }
    pages_scan(s, fine && part && !lost ? 1 : 0, 0);
    cluster_sync(rank == 0);
    const int32_t need = cluster_load(&s.need[kPgThreads], 0);
    int32_t found = 0;
    if (need > 0)
        found = pages_find(p, s, rank, need, [&](int32_t r, int32_t page) {
            p.tail[r] = page;
            p.refs[page] = 1;
        });
    cluster_sync(need > 0);                                       // the tails are written, `used` has been read
    if (rank == 0 && f < p.forks) {
        const bool got = fine && s.need[f + 1] <= found;  // (forks behind the last page that there is need it too, or a later one)
        if (fine && !got)
            bits = SVP_DEV_NO_PAGES;
        if (got && lost)
            bits = SVP_DEV_BAD_CONTEXT;                   // (passed on as -1, without a page)
        const int32_t page = got && part && !lost ? __ldcg(p.tail + s.need[f]) : -1;
        p.plan[f] = make_int4(from, to, got ? whole : -1, page);
        if (got)
            p.used[to] = whole + (part ? 1 : 0);
        if (bits)
            set_status(p.status, bits);
    }
}

constexpr int kPgCopyThreads = 256;

// Copies a page's rows (head, token) in 16-byte pieces, tokens below `tokens` of each head.  A row has a power of two
// of pieces, a page one of tokens.
__device__ __forceinline__ void pages_copy(const PagesCaches &c, void *pool, int32_t from, int32_t to, int32_t tokens,
                                           int32_t page_shift)
{
    constexpr int U = 8;
    const uint8_t *src = static_cast<const uint8_t *>(pool) + from * c.s_page;
    uint8_t *dst = static_cast<uint8_t *>(pool) + to * c.s_page;
    const int32_t count = c.hkv << (page_shift + c.row_shift);
    for (int32_t x0 = threadIdx.x; x0 < count; x0 += U * kPgCopyThreads) {
        uint4 v[U];
        int64_t at[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int32_t x = x0 + u * kPgCopyThreads, y = x >> c.row_shift;
            const int32_t h = y >> page_shift, t = y - (h << page_shift);
            at[u] = x < count && t < tokens ? h * c.s_head + t * c.s_tok + (x - (y << c.row_shift)) * 16 : -1;
            if (at[u] >= 0)
                v[u] = *reinterpret_cast<const uint4 *>(src + at[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (at[u] >= 0)
                *reinterpret_cast<uint4 *>(dst + at[u]) = v[u];
    }
}

// Block (f, y): y = 0 the table's row of fork f, else K (odd y) or V of cache (y - 1) / 2.
__global__ void __launch_bounds__(kPgCopyThreads) pages_fork_copy_kernel(const __grid_constant__ PagesParams p,
                                                                         const __grid_constant__ PagesCaches c)
{
    griddep_launch_dependents();
    griddep_wait();
    const int32_t f = blockIdx.x, tid = threadIdx.x;
    const int4 plan = p.plan[f];
    const int32_t whole = plan.z, page = plan.w;
    if (whole < 0)
        return;
    const int32_t *row = p.table + (int64_t)plan.x * p.max_pages;
    if (blockIdx.y == 0) {
        int32_t *to = p.table + (int64_t)plan.y * p.max_pages;
        if (plan.x == plan.y)
            return;                                       // (nothing of an empty request)
        for (int32_t j = tid; j < p.max_pages; j += kPgCopyThreads) {
            int32_t id = j == whole ? page : -1;
            if (j < whole) {
                id = row[j];
                if (id >= 0 && id < p.num_pages) {
                    atomicAdd(p.refs + id, 1);
                } else {
                    id = -1;
                    set_status(p.status, SVP_DEV_BAD_CONTEXT);
                }
            }
            to[j] = id;
        }
        return;
    }
    if (page < 0)
        return;
    const int32_t from = row[whole], part = __ldg(p.length + f) & ((1 << p.page_shift) - 1);
    if (from < 0 || from >= p.num_pages)
        return;                                           // (never, but for a table that changes meanwhile)
    const int32_t x = (blockIdx.y - 1) >> 1;
    const bool v = (blockIdx.y - 1) & 1;
    pages_copy(c, v ? c.v[x] : c.k[x], from, page, part, p.page_shift);
    uint8_t *exps = v ? c.v_exp[x] : c.k_exp[x];
    if (exps)
        for (int32_t y = tid; y < c.hkv * part; y += kPgCopyThreads) {
            const int32_t h = y / part, t = y - h * part;
            exps[((((int64_t)page * c.hkv) + h) << p.page_shift) + t] = exps[((((int64_t)from * c.hkv) + h) << p.page_shift) + t];
        }
}

// ------------------------------------------------------------------ compact
__global__ void __cluster_dims__(kPgCluster, 1, 1) __launch_bounds__(kPgThreads)
    pages_compact_kernel(const __grid_constant__ PagesParams p)
{
    __shared__ PagesShared s;
    griddep_launch_dependents();
    griddep_wait();
    const uint32_t rank = cluster_rank();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // every warp of the cluster has a run of pages, a multiple of 32
    const int64_t run = (((int64_t)p.num_pages + kPgCluster * kPgWarps * 32 - 1) / (kPgCluster * kPgWarps * 32)) * 32;
    const int64_t lo = min((int64_t)p.num_pages, ((int64_t)rank * kPgWarps + warp) * run);
    const int64_t hi = min((int64_t)p.num_pages, lo + run);
    auto used_at = [&](int64_t page) { return page < hi && __ldcg(p.refs + page) != 0; };
    auto block_sum = [&](int32_t x, int32_t &before) {    // of one value a warp; and of the warps before this one
        __syncthreads();
        if (lane == 0)
            s.warp[warp] = x;
        __syncthreads();
        int32_t v = s.warp[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o)
                v += u;
        }
        const int32_t ahead = __shfl_sync(0xffffffffu, v, (warp + 31) & 31);
        before = warp == 0 ? 0 : ahead;
        return __shfl_sync(0xffffffffu, v, 31);
    };
    int32_t in_use = 0, before_warp, before_block;
#pragma unroll 4
    for (int64_t x = lo; x < hi; x += 32)
        in_use += __popc(__ballot_sync(0xffffffffu, used_at(x + lane)));
    const int32_t mine = block_sum(in_use, before_warp);
    const int32_t live = pages_total(s, rank, 0, mine, before_block);
    // pages in use before this warp's run; with L of them, the free ones before page x < L are x less
    // those in use before it, and the ones in use at L or behind, those before x less those before L
    const int32_t before = before_block + before_warp;
    // in use before L: the warp whose run holds L (or whose run ends the pool there) counts them
    int32_t below = 0;
    if (live >= lo && live < hi)
        for (int64_t x = lo; x < live; x += 32)
            below += __popc(__ballot_sync(0xffffffffu, x + lane < live && used_at(x + lane)));
    int32_t unused_before, unused_block;
    const bool holds = live >= lo && live < hi;
    const int32_t below_all = pages_total(s, rank, 1, block_sum(holds ? before + below : 0, unused_before), unused_block);
    const int32_t used_below = live >= p.num_pages ? live : below_all;
    const int32_t most = p.num_pages / 2 + 1;
    int32_t ahead = before;
    for (int64_t x = lo; x < hi; x += 32) {
        const int64_t page = x + lane;
        const uint32_t mask = __ballot_sync(0xffffffffu, used_at(page));
        const int32_t used_before = ahead + __popc(mask & ((1u << lane) - 1u));
        if (page < hi) {
            // (places below `most` but for counts that change meanwhile)
            const int32_t hole = (int32_t)page - used_before, mover = used_before - used_below;
            if (page < live && !(mask >> lane & 1u) && (uint32_t)hole < (uint32_t)most)
                p.holes[hole] = (int32_t)page;
            if (page >= live && (mask >> lane & 1u) && (uint32_t)mover < (uint32_t)most) {
                p.movers[mover] = (int32_t)page;
                p.rank[page] = mover;
            }
        }
        ahead += __popc(mask);
    }
    if (rank == 0 && threadIdx.x == 0) {
        p.moves[0] = min(max(live - used_below, 0), most);
        p.moves[1] = live;
        if (p.live)
            *p.live = live;
    }
    cluster_sync(false);                                       // (no block leaves while another reads its counts)
}

__global__ void __launch_bounds__(kPgCopyThreads) pages_move_kernel(const __grid_constant__ PagesParams p,
                                                                    const __grid_constant__ PagesCaches c)
{
    griddep_launch_dependents();
    griddep_wait();
    const int32_t tid = threadIdx.x;
    const int32_t moves = p.moves[0], live = p.moves[1];
    // (without moves too: an entry at or behind `live` is reported all the same)
    for (int32_t i = blockIdx.x; i < p.n; i += gridDim.x) {
        const int32_t held = p.used[i];
        int32_t *row = p.table + (int64_t)i * p.max_pages;
        for (int32_t j = tid; j < min(held, p.max_pages); j += kPgCopyThreads) {
            const int32_t id = row[j];
            if (id < live || id >= p.num_pages)
                continue;
            const int32_t k = p.rank[id];                 // (old or foreign contents if the page is no mover)
            if (k >= 0 && k < moves && p.movers[k] == id)
                row[j] = p.holes[k];
            else
                set_status(p.status, SVP_DEV_BAD_CONTEXT);
        }
    }
    auto inside = [&](int32_t from, int32_t to) {         // (always, but for counts that changed meanwhile)
        return (uint32_t)from < (uint32_t)p.num_pages && (uint32_t)to < (uint32_t)p.num_pages && from >= live && to < live;
    };
    for (int32_t k = blockIdx.x * kPgCopyThreads + tid; k < moves; k += gridDim.x * kPgCopyThreads) {
        const int32_t from = p.movers[k], to = p.holes[k];
        if (inside(from, to)) {
            p.refs[to] = p.refs[from];
            p.refs[from] = 0;
        }
    }
    const int64_t items = (int64_t)moves * 2 * c.count;
    for (int64_t x = blockIdx.x; x < items; x += gridDim.x) {
        const int32_t k = (int32_t)(x / (2 * c.count)), y = (int32_t)(x - (int64_t)k * 2 * c.count);
        const int32_t from = p.movers[k], to = p.holes[k];
        if (!inside(from, to))
            continue;
        const bool v = y & 1;
        pages_copy(c, v ? c.v[y >> 1] : c.k[y >> 1], from, to, 1 << p.page_shift, p.page_shift);
        uint8_t *exps = v ? c.v_exp[y >> 1] : c.k_exp[y >> 1];
        if (exps) {
            const int32_t bytes = c.hkv << p.page_shift;  // (a multiple of 16)
            for (int32_t z = tid * 16; z < bytes; z += kPgCopyThreads * 16)
                *reinterpret_cast<uint4 *>(exps + (int64_t)to * bytes + z) =
                    *reinterpret_cast<const uint4 *>(exps + (int64_t)from * bytes + z);
        }
    }
}

// ------------------------------------------------------------------ host side
int sm_count();

static size_t up256(size_t x) { return (x + 255) / 256 * 256; }

struct PagesWs {
    size_t plan, tail, holes, movers, rank, bytes;
};

static PagesWs pages_ws(int64_t num_pages)
{
    // (at most half of the pages move, to as many holes)
    const size_t half = up256((size_t)(num_pages / 2 + 1) * 4);
    PagesWs w;
    w.plan = kWsHeader + 256;                             // (the moves' number between)
    w.tail = w.plan + kPgRequests * sizeof(int4);
    w.holes = w.tail + kPgRequests * 4;
    w.movers = w.holes + half;
    w.rank = w.movers + half;
    w.bytes = w.rank + up256((size_t)num_pages * 4);
    return w;
}

static svp_status pages_params(const svp_pages *pages, PagesParams &p)
{
    if (!pages || pages->n < 0 || pages->max_pages < 0 || pages->num_pages < 0 || pages->num_pages >= ((int64_t)1 << 31))
        return SVP_EINVAL;
    if (pages->page_size != 16 && pages->page_size != 32 && pages->page_size != 64 && pages->page_size != 128)
        return SVP_EUNSUPPORTED;
    if (pages->n > kPgRequests || (int64_t)pages->max_pages * pages->page_size >= ((int64_t)1 << 31) ||
        (int64_t)pages->n * pages->max_pages >= ((int64_t)1 << 31))
        return SVP_EUNSUPPORTED;
    p.table = pages->block_table;
    p.used = pages->used;
    p.refs = pages->refs;
    p.n = pages->n;
    p.max_pages = pages->max_pages;
    p.num_pages = (int32_t)pages->num_pages;
    p.page_shift = pages->page_size == 16 ? 4 : pages->page_size == 32 ? 5 : pages->page_size == 64 ? 6 : 7;
    return SVP_OK;
}

static bool pages_there(const PagesParams &p)            // (an empty tensor has no address)
{
    return (p.used || p.n == 0) && (p.table || p.n == 0 || p.max_pages == 0) && (p.refs || p.num_pages == 0);
}

static svp_status pages_workspace(void *ws, size_t ws_bytes, PagesParams &p)
{
    const PagesWs w = pages_ws(p.num_pages);
    if (!ws || ws_bytes < w.bytes)
        return SVP_EWORKSPACE;
    if (reinterpret_cast<uintptr_t>(ws) & 15)
        return SVP_EINVAL;
    uint8_t *b = static_cast<uint8_t *>(ws);
    p.status = reinterpret_cast<int32_t *>(b);
    p.moves = reinterpret_cast<int32_t *>(b + kWsHeader);
    p.plan = reinterpret_cast<int4 *>(b + w.plan);
    p.tail = reinterpret_cast<int32_t *>(b + w.tail);
    p.holes = reinterpret_cast<int32_t *>(b + w.holes);
    p.movers = reinterpret_cast<int32_t *>(b + w.movers);
    p.rank = reinterpret_cast<int32_t *>(b + w.rank);
    return SVP_OK;
}

static svp_status pages_caches(const svp_pages *pages, const svp_cache *caches, int32_t count, int32_t hkv, int32_t d,
                               PagesCaches &c)
{
    if (count < 0 || (count > 0 && !caches))
        return SVP_EINVAL;
    if (count > SVP_PAGES_MAX_CACHES || (count > 0 && hkv > 4096))
        return SVP_EUNSUPPORTED;
    std::memset(&c, 0, sizeof c);
    c.count = count;
    for (int32_t x = 0; x < count; ++x) {
        CacheParams cp{};
        const svp_status st = cache_params(caches + x, hkv, d, cp);
        if (st != SVP_OK)
            return st;
        if (caches[x].page_size != pages->page_size || caches[x].num_pages != pages->num_pages ||
            caches[x].dtype != caches[0].dtype || cp.s_page != caches[0].stride_page ||
            cp.s_head != caches[0].stride_head || cp.s_tok != caches[0].stride_tok)
            return SVP_EINVAL;
        c.k[x] = cp.k;
        c.v[x] = cp.v;
        if (caches[x].dtype == SVP_E4M3) {
            c.k_exp[x] = cp.k_exp;
            c.v_exp[x] = cp.v_exp;
        }
    }
    if (count > 0) {
        const int64_t esz = caches[0].dtype == SVP_F32 ? 4 : caches[0].dtype == SVP_BF16 ? 2 : 1;
        c.s_page = caches[0].stride_page * esz;
        c.s_head = caches[0].stride_head * esz;
        c.s_tok = caches[0].stride_tok * esz;
        c.hkv = hkv;
        while ((16 << c.row_shift) < d * esz)
            ++c.row_shift;
    }
    return SVP_OK;
}

}  // namespace svp

using namespace svp;

extern "C" {

svp_status svp_pages_workspace_size(const svp_pages *pages, size_t *bytes)
{
    PagesParams p{};
    if (!bytes)
        return SVP_EINVAL;
    const svp_status st = pages_params(pages, p);
    if (st == SVP_OK)
        *bytes = pages_ws(p.num_pages).bytes;
    return st;
}

svp_status svp_pages_resize(const svp_pages *pages, const int32_t *length, void *ws, size_t ws_bytes, void *stream)
{
    PagesParams p{};
    svp_status st = pages_params(pages, p);
    if (st != SVP_OK)
        return st;
    st = pages_workspace(ws, ws_bytes, p);
    if (st != SVP_OK)
        return st;
    if (p.n == 0)
        return SVP_OK;
    if (!pages_there(p) || !length)
        return SVP_EINVAL;
    p.length = length;
    return launch_pdl(pages_resize_kernel, dim3(kPgCluster), dim3(kPgThreads), 0, (cudaStream_t)stream, p) == cudaSuccess
               ? SVP_OK
               : SVP_ECUDA;
}

svp_status svp_pages_fork(const svp_pages *pages, const svp_cache *caches, int32_t n_caches, int32_t hkv, int32_t d,
                          const int32_t *src, const int32_t *dst, const int32_t *length, int32_t forks, void *ws,
                          size_t ws_bytes, void *stream)
{
    PagesParams p{};
    PagesCaches c;
    svp_status st = pages_params(pages, p);
    if (st != SVP_OK)
        return st;
    st = pages_caches(pages, caches, n_caches, hkv, d, c);
    if (st != SVP_OK)
        return st;
    if (forks < 0)
        return SVP_EINVAL;
    if (forks > kPgRequests)
        return SVP_EUNSUPPORTED;
    st = pages_workspace(ws, ws_bytes, p);
    if (st != SVP_OK)
        return st;
    if (p.n == 0 || forks == 0)
        return SVP_OK;
    if (!pages_there(p) || !src || !dst || !length)
        return SVP_EINVAL;
    p.src = src;
    p.dst = dst;
    p.length = length;
    p.forks = forks;
    if (launch_pdl(pages_fork_kernel, dim3(kPgCluster), dim3(kPgThreads), 0, (cudaStream_t)stream, p) != cudaSuccess)
        return SVP_ECUDA;
    return launch_pdl(pages_fork_copy_kernel, dim3((unsigned)forks, (unsigned)(1 + 2 * n_caches)), dim3(kPgCopyThreads), 0,
                      (cudaStream_t)stream, p, c) == cudaSuccess
               ? SVP_OK
               : SVP_ECUDA;
}

svp_status svp_pages_compact(const svp_pages *pages, const svp_cache *caches, int32_t n_caches, int32_t hkv, int32_t d,
                             int32_t *live, void *ws, size_t ws_bytes, void *stream)
{
    PagesParams p{};
    PagesCaches c;
    svp_status st = pages_params(pages, p);
    if (st != SVP_OK)
        return st;
    st = pages_caches(pages, caches, n_caches, hkv, d, c);
    if (st != SVP_OK)
        return st;
    st = pages_workspace(ws, ws_bytes, p);
    if (st != SVP_OK)
        return st;
    if (!pages_there(p))
        return SVP_EINVAL;
    p.live = live;
    if (launch_pdl(pages_compact_kernel, dim3(kPgCluster), dim3(kPgThreads), 0, (cudaStream_t)stream, p) != cudaSuccess)
        return SVP_ECUDA;
    return launch_pdl(pages_move_kernel, dim3((unsigned)(sm_count() * 8)), dim3(kPgCopyThreads), 0, (cudaStream_t)stream, p,
                      c) == cudaSuccess
               ? SVP_OK
               : SVP_ECUDA;
}

}  // extern "C"
