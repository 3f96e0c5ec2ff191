// prefix_pieces.cuh -- how the work of svp_prefix_attn is cut: the sequence of pairs of chunk_pieces.cuh with
// the groups that share a beginning in front of the requests.
//
// A shared group is one more "request": its rows are those of all its requests, which lie side by side, its
// keys the P positions that they have in common, seen by every row.  Its requests come after all groups and
// have the keys from P on.  So both kinds are split over the CTAs together, and a group's pages are read
// once for as many rows as a block takes (256 / G tokens) instead of once a request.
//
// A group is shared where that saves a pass: where its rows fill fewer blocks together than apart (two
// requests at least, and not prompts that fill their own blocks), P taken down to whole pages.  Else, or where
// the group's numbers are not in order, its requests have all their keys themselves.
#pragma once

#include "chunk_pieces.cuh"

namespace svp {

constexpr int kPxMost = 1024;         // requests, and groups, of a call

// One sequence of all pairs, or one of the groups and one of the requests, each with blocks of its own (prefix_tc.cu
// says when).
enum { kPxAll = 0, kPxBeside = 1 };
// Rows of a KV head up to which requests have blocks of their own.  One block of 8 in warp-level products; with 16 rows
// they took 136 us where the tile kernel's pairs take 126 (64 requests of 4 tokens behind 16384, bf16; 8-bit
// 209 and 187).
constexpr int kPxRows = 8;

// What the joining kernel needs of a request, and of its group, written by the first CTA of the kernel that has the pairs.
struct PrefixRec {
    int32_t off, k, L, P;             // first row, rows, cached tokens behind the P common ones (k 0: skipped)
    int64_t base;                     // cost before its pairs
};
struct PrefixGroup {
    int32_t off, k;                   // first row and rows
    int64_t base;
};

// Costs of a key: a request's pair of one query tile, and a pair of two.  In the tile kernel a request's few tiles of its
// own take longer than those of a long stream (64 requests of 8 rows, 64 to 2048 own tokens: 2.2 us each, where a group's
// take 1.4, or 1.9 for two query tiles).  64 requests of 4 and of 8 rows behind 16384, us with 3 : 4, 4 : 5 and 4 : 4: bf16
// 126 and 188, 118 and 180, 118 and 193; 8-bit 183 and 266, 174 and 259, 160 and 257.  Where nothing is shared the costs,
// and so the pieces, are svp_chunk_attn's.
struct PxCosts {
    int32_t one, two;
};

__device__ __forceinline__ PxCosts px_costs(int32_t part, bool shared, bool q8)
{
    static_assert(kShortCost == 3 && kLongCost == 4 && kMostCost == 5, "px_tile_at");
    return part == kPxAll && shared ? PxCosts{4, q8 ? 4 : kMostCost} : PxCosts{kShortCost, kLongCost};
}

struct PrefixPiece : ChunkPiece {     // i: place in the sequence of groups and requests
    int32_t ne, ng;                   // length of the sequence, and groups in it
    const int4 *plan;                 // this CTA's copy: (first row, rows, P, row of the block table), then (first
                                      // row, rows, tokens behind P, P)
    int32_t row, first;               // row of the block table, and the first key's position
    int32_t R;                        // tokens of a query tile
    PxCosts cost;
    bool group;
};

__device__ __forceinline__ int64_t ck_table(const ChunkParams &p, const PrefixPiece &s)
{
    return (int64_t)s.row * p.c.max_pages + (s.first >> p.c.page_shift);
}
__device__ __forceinline__ int32_t ck_last(const PrefixPiece &s, int32_t tok)
{
    return s.group ? s.L - 1 : s.L + s.tb0 + tok;
}
__device__ __forceinline__ bool ck_kept(const PrefixPiece &s) { return s.group || s.first > 0; }

__device__ __forceinline__ int32_t px_weight(int32_t nt, int32_t one, int32_t two, int32_t k, int32_t R)   // nt query tiles a block
{
    return nt == 2 && k > R ? two : one;
}

__device__ __forceinline__ int32_t px_tile_at(int64_t x, int32_t wt)   // ck_tile_at for the costs 3, 4 and 5
{
    const int64_t s = (int64_t)kStartKeys * wt;
    if (x <= s)
        return 0;
    const uint32_t y = (uint32_t)((x - s - 1) / kCkKeys);
    return (int32_t)(wt == 3 ? y / 3u : wt == 4 ? y / 4u : y / 5u) + 1;
}

// Keys of one KV head of a group of k rows, B a block: each block sees all L.
__device__ __forceinline__ int64_t px_head_keys(int32_t L, int32_t k, int32_t B)
{
    return (int64_t)((k + B - 1) / B) * ((int64_t)kStartKeys + L);
}

template <int NT>
__device__ __forceinline__ bool ck_set(const ChunkParams &p, PrefixPiece &s, int64_t v1, int32_t t0)
{
    const int32_t B = NT * s.R;
    s.tb0 = s.b * B;
    s.ntok = min(B, s.k - s.tb0);
    s.len = s.group ? s.L : s.L + s.tb0 + s.ntok;
    s.nt = (s.len + kCkKeys - 1) / kCkKeys;
    s.t0 = t0;
    const int32_t wt = s.wt;
    const int64_t y = v1 - s.base;
    s.t1 = y >= (int64_t)wt * (kStartKeys + (int64_t)s.len) ? s.nt : min(s.nt, px_tile_at(y, wt));
    return s.t0 < s.t1;
}

template <int NT>
__device__ __forceinline__ bool px_entry(const ChunkParams &p, PrefixPiece &s, const int4 x)
{
    const int32_t B = NT * s.R;
    s.group = s.i < s.ng;
    s.off = x.x;
    s.k = x.y;
    s.L = x.z;
    s.row = s.group ? x.w : s.i - s.ng;
    s.first = s.group ? 0 : x.w;
    if (s.k <= 0)
        return false;
    s.nb = (s.k + B - 1) / B;
    s.wt = px_weight(NT, s.group ? kShortCost : s.cost.one, s.cost.two, s.k, s.R);
    return true;
}

__device__ __forceinline__ int32_t px_slot(const PrefixPiece &s) { return s.i < s.ng ? s.i : kPxMost + s.i - s.ng; }

template <int NT>
__device__ __forceinline__ bool ck_request(const ChunkParams &p, PrefixPiece &s)
{
    return px_entry<NT>(p, s, __ldcg(s.plan + px_slot(s)));
}

template <int NT>
__device__ __forceinline__ bool ck_next(const ChunkParams &p, PrefixPiece &s, int64_t v1)
{
    s.base += (int64_t)s.wt * (kStartKeys + (int64_t)s.len);
    if (s.base >= v1)
        return false;
    if (++s.b == s.nb) {
        s.b = 0;
        if (++s.g == p.c.hkv) {
            s.g = 0;
            do {
                if (++s.i >= s.ne)
                    return false;     // (never: base < v1 <= the total)
            } while (!ck_request<NT>(p, s));
        }
    }
    return ck_set<NT>(p, s, v1, 0);
}

// Shared memory of the prologue, where the ring (96 KB at least) is later.
struct PrefixSums {
    int64_t prefix[2 * kPxMost + 1];
    int4 plan[2 * kPxMost];           // as the CTA's copy in the workspace
    int32_t cu[kPxMost + 1], gcu[kPxMost + 1], len[kPxMost], ctx[kPxMost];
    int32_t blocks[kPxMost];          // blocks that the group's requests fill apart
    int32_t bad[kPxMost];
    int32_t lead[kPxMost];            // its first request with rows
    int32_t shared[kPxMost];          // tokens that it shares, 0: none
    int32_t gbase[kPxMost];           // its place in the sequence
    unsigned long long longs;         // cost of the groups with two query tiles a block
    int32_t broken, groups_broken, any_shared;
    int32_t cnt[32];
    int64_t tot[32];
};

// Exclusive sums of cost (and of 0 / 1 counts) over the block's threads, chunk by chunk.
struct PrefixScan {
    int64_t running;
    int32_t count;
};

__device__ __forceinline__ void px_scan(PrefixSums &x, PrefixScan &run, int64_t cost, bool one, int64_t &before, int32_t &place)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarp = blockDim.x >> 5;
    int64_t incl = cost;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o)
            incl += v;
    }
    const uint32_t ones = __ballot_sync(0xffffffffu, one);
    __syncthreads();                  // (the sums of the chunk before have been read)
    if (lane == 31)
        x.tot[warp] = incl;
    if (lane == 0)
        x.cnt[warp] = __popc(ones);
    __syncthreads();
    int64_t t = lane < nwarp ? x.tot[lane] : 0;
    int32_t c = lane < nwarp ? x.cnt[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, t, o);
        const int32_t u = __shfl_up_sync(0xffffffffu, c, o);
        if (lane >= o) {
            t += v;
            c += u;
        }
    }
    const int64_t ahead = __shfl_sync(0xffffffffu, t, (warp + 31) & 31);
    const int32_t ahead_c = __shfl_sync(0xffffffffu, c, (warp + 31) & 31);
    before = run.running + incl - cost + (warp == 0 ? 0 : ahead);
    place = run.count + __popc(ones & ((1u << lane) - 1u)) + (warp == 0 ? 0 : ahead_c);
    run.running += __shfl_sync(0xffffffffu, t, 31);
    run.count += __shfl_sync(0xffffffffu, c, 31);
}

// Cost before each of the sequence's groups and requests into x->prefix, their places and sizes into x->plan and this
// CTA's copy, and (first CTA) what the joining kernel needs.  Returns the sequence's length.
template <int NT>
__device__ __forceinline__ int32_t px_prologue(const ChunkParams &p, void *smem, int32_t part, bool q8)
{
    PrefixSums &x = *static_cast<PrefixSums *>(smem);
    const int32_t tid = threadIdx.x, nt = blockDim.x, B = NT * p.R, OB = p.own_NT * p.own_R, n = p.n, ng = p.ng;
    const bool tells = blockIdx.x == 0;
    int4 *plan = p.plan + (int64_t)blockIdx.x * 2 * kPxMost;
    if (tid == 0) {
        x.broken = x.groups_broken = x.any_shared = 0;
        x.longs = 0;
    }
    // everything that is read, in one round trip
    for (int32_t i = tid; i <= n; i += nt) {
        x.cu[i] = __ldg(p.cu + i);
        if (i < n)
            x.ctx[i] = __ldg(p.ctx_len + i);
    }
    for (int32_t g = tid; g <= ng; g += nt) {
        x.gcu[g] = __ldg(p.cu_groups + g);
        if (g < ng) {
            x.len[g] = __ldg(p.prefix_len + g);
            x.blocks[g] = x.bad[g] = 0;
            x.lead[g] = n;
        }
    }
    __syncthreads();
    // request i's group, or -1 (the group's bounds are looked at beside)
    auto group_of = [&](int32_t i) -> int32_t {
        if (i < x.gcu[0] || i >= x.gcu[ng])
            return -1;
        int32_t lo = 0, hi = ng;
        while (hi - lo > 1) {
            const int32_t mid = (lo + hi) >> 1;
            if (x.gcu[mid] <= i)
                lo = mid;
            else
                hi = mid;
        }
        return lo;
    };
    for (int32_t g = tid; g < ng; g += nt)
        if (x.gcu[g] < 0 || x.gcu[g + 1] < x.gcu[g] || x.gcu[g + 1] > n)
            x.groups_broken = 1;
    for (int32_t i = tid; i < n; i += nt) {
        const int32_t off = x.cu[i], end = x.cu[i + 1], L = x.ctx[i], k = end - off;
        if (off < 0 || end < off || end > p.m_cap)
            x.broken = 1;
        if (off < 0 || end <= off)
            continue;
        const int32_t bad = ck_bad(p, off, end, L), g = group_of(i);
        if (bad && tells)
            set_status(p.status, bad);
        if (g >= 0) {
            if (!bad && x.len[g] > L && tells)
                set_status(p.status, SVP_DEV_BAD_CONTEXT);
            if (bad || x.len[g] > L)
                x.bad[g] = 1;
            atomicAdd(&x.blocks[g], bad ? 0 : (k + p.share_rows - 1) / p.share_rows);
            atomicMin(&x.lead[g], i);
        }
    }
    __syncthreads();
    const bool broken = x.broken != 0, grouped = x.groups_broken == 0 && !broken;
    if (tells && tid == 0 && (broken || x.groups_broken))
        set_status(p.status, SVP_DEV_BAD_SLOTS);
    for (int32_t g = tid; g < ng; g += nt) {
        int32_t P = 0;
        if (grouped) {
            const int32_t k = x.cu[x.gcu[g + 1]] - x.cu[x.gcu[g]];
            if (x.len[g] < 0 && tells)
                set_status(p.status, SVP_DEV_BAD_CONTEXT);
            if (!x.bad[g] && x.len[g] > 0 && k > 0 && (k + p.share_rows - 1) / p.share_rows < x.blocks[g])
                P = x.len[g] >> p.c.page_shift << p.c.page_shift;
        }
        x.shared[g] = P;
        if (P > 0)
            x.any_shared = 1;
    }
    __syncthreads();
    const PxCosts cs = px_costs(part, x.any_shared != 0, q8);
    // the groups and the requests in one sequence of sums; the requests' places follow when the number of groups is known
    const int32_t to = ng + n;
    PrefixScan run{0, 0};
    for (int32_t e0 = 0; e0 < to; e0 += nt) {
        const int32_t e = e0 + tid;
        int64_t cost = 0;
        int4 what = make_int4(0, 0, 0, 0);
        bool one = false;
        if (e < to && !broken) {
            if (e < ng) {
                one = x.shared[e] > 0;                    // (else its bounds may be anything)
                if (one) {
                    what = make_int4(x.cu[x.gcu[e]], x.cu[x.gcu[e + 1]] - x.cu[x.gcu[e]], x.shared[e], x.lead[e]);
                    cost = px_head_keys(what.z, what.y, B) * px_weight(NT, kShortCost, cs.two, what.y, p.R) * p.c.hkv;
                    if (NT == 2 && what.y > p.R)
                        atomicAdd(&x.longs, (unsigned long long)cost);
                }
            } else {
                const int32_t i = e - ng, off = x.cu[i], k = x.cu[i + 1] - off, L = x.ctx[i];
                if (k > 0 && !ck_bad(p, off, x.cu[i + 1], L)) {
                    const int32_t g = grouped ? group_of(i) : -1, P = g >= 0 ? x.shared[g] : 0;
                    what = make_int4(off, k, L - P, P);
                    cost = ck_head_keys(what.z, k, OB) * px_weight(p.own_NT, cs.one, cs.two, k, p.own_R) * p.c.hkv;
                }
            }
        }
        int64_t before;
        int32_t at;
        px_scan(x, run, cost, one, before, at);
        if (e < ng) {
            if (one) {
                x.prefix[at] = before;
                x.plan[at] = what;
                plan[at] = what;
                x.gbase[e] = at;
            }
        } else if (e < to) {
            // (kept where groups cannot reach until all are counted: shifted below)
            const int32_t i = e - ng;
            x.plan[kPxMost + i] = what;
            plan[kPxMost + i] = what;
            x.prefix[kPxMost + i] = before;
            if (tells)
                p.rec[i] = PrefixRec{what.x, what.y, what.z, what.w, before};
        }
    }
    const int32_t length = run.count + n;
    if (tid == 0)
        x.prefix[2 * kPxMost] = run.running;
    __syncthreads();
    if (tells && tid == 0) {
        p.total[0] = run.running;
        p.total[1] = x.prefix[kPxMost];                   // (of the groups)
        p.total[2] = (int64_t)x.longs;
        p.total[3] = x.any_shared;
    }
    if (tells)
        for (int32_t i = tid; i < n; i += nt) {
            const int32_t g = grouped ? group_of(i) : -1;
            PrefixGroup gr{0, 0, 0};
            if (g >= 0 && x.shared[g] > 0) {
                const int32_t at = x.gbase[g];
                gr = PrefixGroup{x.plan[at].x, x.plan[at].y, x.prefix[at]};
            }
            p.grp[i] = gr;
        }
    return length;
}

__device__ __forceinline__ int64_t px_total(const PrefixSums &x, int32_t) { return x.prefix[2 * kPxMost]; }
__device__ __forceinline__ int64_t px_total(const int64_t *prefix, int32_t n) { return prefix[n]; }

// Cost before entry i of a sequence of ne with ng groups.
__device__ __forceinline__ int64_t px_before(const PrefixSums &x, int32_t ng, int32_t ne, int32_t i)
{
    return x.prefix[i == ne ? 2 * kPxMost : i < ng ? i : kPxMost + i - ng];
}

template <int NT>
__device__ __forceinline__ bool ck_first(const ChunkParams &p, const PrefixSums &x, PrefixPiece &s, int64_t v0, int64_t v1)
{
    if (v0 >= v1)
        return false;
    const int32_t B = NT * s.R;
    int32_t lo = 0, hi = s.ne;
    while (hi - lo > 1) {             // last pairs with prefix <= v0 (they have a cost: v0 < total)
        const int32_t mid = (lo + hi) >> 1;
        if (px_before(x, s.ng, s.ne, mid) <= v0)
            lo = mid;
        else
            hi = mid;
    }
    s.i = lo;
    px_entry<NT>(p, s, x.plan[px_slot(s)]);
    const int64_t start = px_before(x, s.ng, s.ne, lo);
    const int32_t wt = s.wt, slope = s.group ? 0 : B;
    const int64_t H = (s.group ? px_head_keys(s.L, s.k, B) : ck_head_keys(s.L, s.k, B)) * wt;
    int64_t rem = v0 - start;
    s.g = (int32_t)(rem / H);
    rem -= s.g * H;
    // last block with cost before it <= rem (chunk_pieces.cuh; a group's blocks cost the same each)
    const int64_t a = (int64_t)kStartKeys + s.L;
    int64_t b;
    if (s.group) {
        b = rem / (a * wt);
    } else {
        const float h = (float)a + 0.5f * B;
        b = (int64_t)((sqrtf(h * h + 2.0f * B * ((float)rem / wt)) - h) / B);
    }
    b = b < 0 ? 0 : b > s.nb - 1 ? s.nb - 1 : b;
    while (b + 1 < s.nb && ck_before(a, slope, b + 1) * wt <= rem)
        ++b;
    while (b > 0 && ck_before(a, slope, b) * wt > rem)
        --b;
    s.b = (int32_t)b;
    s.base = start + s.g * H + ck_before(a, slope, b) * wt;
    const int32_t t0 = px_tile_at(v0 - s.base, wt);
    const bool have = ck_set<NT>(p, s, v1, t0);
    return have || (t0 >= s.nt && ck_next<NT>(p, s, v1));
}

__device__ __forceinline__ void px_bind(const ChunkParams &p, const PrefixSums &x, PrefixPiece &s, int32_t length, int32_t part, bool q8)
{
    s.cost = px_costs(part, x.any_shared != 0, q8);
    s.plan = p.plan + (int64_t)blockIdx.x * 2 * kPxMost;
    s.ne = length;
    s.ng = length - p.n;
    s.R = p.R;
}

// kPxBeside: of `ctas` blocks, those that the groups have; the others have the requests.  all: cost of both, groups: of
// the groups, which come first in the sums, longs: of those with two query tiles a block.  In ns a unit, 64 tokens
// behind prefixes of 16384 (two tiles) and 4 x 20480 (one), with 0 to 1024 of their own: over bf16 pages two tiles 4.0 to
// 4.6, one 3.5, requests 2.8 to 3.1; over 8-bit ones, where tiles are widened for the groups, two 5.4 to 6.3, one 3.9,
// requests 2.5 to 3.7.  So two tiles count 5 / 4 (8-bit 3 / 2), and requests 14 / 16 (12 / 16).
__device__ __forceinline__ int32_t px_split(int64_t all, int64_t groups, int64_t longs, int32_t ctas, bool q8)
{
    if (groups == 0 || groups == all)
        return groups == 0 ? 0 : ctas;
    const int64_t a = 16 * groups + (q8 ? 8 : 4) * longs, b = a + (q8 ? 12 : 14) * (all - groups);
    return max(1, min(ctas - 1, (int32_t)((a * ctas + b / 2) / b)));
}

// Place of (row, head) of a part that one piece has all of, a group's or a request's behind one.
__device__ __forceinline__ int64_t px_place(const ChunkParams &p, bool group, int32_t row, int32_t head)
{
    return ((group ? 0 : (int64_t)p.m_cap) + row) * p.hq + head;
}

}  // namespace svp
