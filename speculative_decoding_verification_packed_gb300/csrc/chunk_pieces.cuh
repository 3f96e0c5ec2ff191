// chunk_pieces.cuh -- how the work of svp_chunk_attn is cut: shared by its tcgen05 kernel, its short
// kernel for 8-bit pages and the kernel that joins split pairs.
#pragma once

#include "svp_cache.cuh"

namespace svp {

constexpr int kCkKeys = 128;          // keys a KV tile
constexpr int kCkSub = 16384;         // [128 rows][64] bf16, 128-byte swizzled
// Cost of starting a pair, in keys.  A prompt of 4096 tokens and 24 blocks of 8 among two prompts of 2048
// (8-bit) take 178 and 332 us with 64, 146 and 325 with 256, 140 and 319 with 512.  (512 was not looked at
// over other calls.)
constexpr int kStartKeys = 256;
// Cost of a key with one query tile, and with two: where 3 to 4 takes 325 us on those blocks and prompts, 2 to
// 3 takes 329 and 1 to 1 345 (the one prompt takes 146 to 147 with each).
constexpr int kShortCost = 3, kLongCost = 4;
// Smallest share of a CTA, more than a tile's cost: a shorter one is not worth its join.  One token over 500
// keys takes 14.6 us, with 2048 16.6 (700 keys 14.6 and 19.0).
constexpr int kShareCost = 640;
// P stays below 2^8 times its value at the reference, but over bf16 pages in a tile that is read once: there it
// may go on as long as a row's sum over the tile is at most 2^15 (chunk_tc.cu).
constexpr float kCkSlack = 8.0f;
// P in fp16 (8-bit pages) is 2^7 at the reference: with the slack it stays below 2^15, and what fp16 cannot
// hold (digits under 2^-24) is 2^-31 of the row's largest probability, so that a million keys lose no weight.
constexpr float kCkLift = 7.0f;

// Query rows of a KV head up to which 8-bit pages take chunk_short.cu.  64 requests x 18000 keys, 8 KV heads,
// d 128, 4 and 16 rows: 363 and 488 us there, 640 and 643 in chunk_tc.cu (d 64, 4 and 16 rows: 330 and 352
// against 571 and 574).  32 rows, in two groups of warps, took 854 us there and take 649 in chunk_tc.cu.
constexpr int kShortRows = 16;

struct ChunkDesc {                    // a pair that was split: read by the joining kernel
    int32_t np, row0, ntok, g;        // pieces (0: none), first packed row, tokens, KV head
};

struct ChunkParams {
    CUtensorMap tm_q, tm_k, tm_v;
    CacheParams c;
    const int32_t *ctx_len, *cu;
    const void *q;                    // [m_cap, hq, d] bf16, rows q_stride apart
    int64_t q_stride;
    int32_t n, m_cap, w, hq, G, R;    // R: tokens of a query tile
    float scale_log2;
    int32_t out32;                    // out is 32-byte aligned
    void *out;
    float *lse;
    int32_t *status;
    ChunkDesc *desc;                  // [grid]
    float2 *part_ml;                  // [2 * grid][rows]
    float *part_o;                    // [2 * grid][rows][d]; rows = 256 (d <= 128) or 128
    int32_t nslot, nraw;              // bf16 tile slots, raw slots (8-bit pages)
    int32_t off_ring, off_raw, off_misc;
    int32_t Rb, qsub;                 // tokens of a query box: min(R, w); bytes of its [rows][64] blocks
};

// One CTA an SM.  A dependent of the previous kernel starts 3 us earlier, but its CTAs go to SMs as these
// fall free, and where neighbours land matters: a CTA with long pieces that shares a TPC with one with
// short pieces takes 12% longer.  So chunk_tc.cu is launched as a dependent in clusters of two, which
// keep neighbours on one TPC (blocks among prompts over 8-bit pages, back to back: 375 us without
// clusters, 322 with; no dependent 327), and chunk_short.cu, which clusters do not help, as one only
// when the call may be short (see there).
inline cudaError_t launch_ctas(void (*kernel)(ChunkParams), int ctas, int threads, size_t smem, cudaStream_t stream,
                               const ChunkParams &p, bool dependent, bool pairs)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    cfg.attrs = attr;
    if (dependent) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (pairs) {                          // (clusters of one are placed otherwise than no clusters)
        attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        attr[cfg.numAttrs].val.clusterDim.x = 2;
        attr[cfg.numAttrs].val.clusterDim.y = attr[cfg.numAttrs].val.clusterDim.z = 1;
        ++cfg.numAttrs;
    }
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

// ------------------------------------------------------------------ the sequence of pairs
struct ChunkPiece {
    int32_t i, g, b, nb;              // request, KV head, token block, blocks of the request
    int32_t off, k, L;                // the request's first packed row, rows, cached tokens
    int32_t tb0, ntok, len;           // first token and tokens of the block; keys it sees
    int32_t nt, t0, t1;               // its KV tiles, and those of this piece
    int32_t wt;                       // cost of a key
    int64_t base;                     // cost before the pair
};

__device__ __forceinline__ int64_t ck_before(int64_t a, int64_t B, int64_t b)   // keys of blocks 0..b-1
{
    return b * a + B * (b * (b + 1) / 2);
}

// A key of a request with blocks of two query tiles costs more (its tile is worked on twice).
template <int NT>
__device__ __forceinline__ int32_t ck_weight(int32_t k, int32_t R)
{
    return NT == 2 && k > R ? kLongCost : kShortCost;
}

// Keys of one KV head of a request: kStartKeys + L + (those of its own tokens) for each block.
__device__ __forceinline__ int64_t ck_head_keys(int32_t L, int32_t k, int32_t B)
{
    const int64_t nb = (k + B - 1) / B, a = (int64_t)kStartKeys + L;
    return nb == 0 ? 0 : ck_before(a, B, nb - 1) + a + k;
}

__device__ __forceinline__ int32_t ck_tile_at(int64_t x, int32_t wt)   // first tile at or after cost x of a pair
{
    const int64_t s = (int64_t)kStartKeys * wt;
    if (x <= s)
        return 0;
    const uint32_t y = (uint32_t)((x - s - 1) / kCkKeys);    // (x is at most a pair's cost: below 2^34)
    return (int32_t)(wt == kShortCost ? y / kShortCost : y / kLongCost) + 1;
}

template <int NT>
__device__ __forceinline__ bool ck_set(const ChunkParams &p, ChunkPiece &s, int64_t v1, int32_t t0)
{
    const int32_t B = NT * p.R;
    s.tb0 = s.b * B;
    s.ntok = min(B, s.k - s.tb0);
    s.len = s.L + s.tb0 + s.ntok;
    s.nt = (s.len + kCkKeys - 1) / kCkKeys;
    s.t0 = t0;
    const int32_t wt = s.wt;
    const int64_t y = v1 - s.base;
    s.t1 = y >= (int64_t)wt * (kStartKeys + (int64_t)s.len) ? s.nt : min(s.nt, ck_tile_at(y, wt));
    return s.t0 < s.t1;
}

// Status bits of a request that breaks the contract.
__device__ __forceinline__ int32_t ck_bad(const ChunkParams &p, int32_t off, int32_t end, int32_t L)
{
    if (off < 0 || end < off || end - off > p.w || end > p.m_cap)
        return SVP_DEV_BAD_SLOTS;
    if (end > off && (L < 0 || (int64_t)L + (end - off) > ((int64_t)p.c.max_pages << p.c.page_shift)))
        return SVP_DEV_BAD_CONTEXT;
    return 0;
}

// Request s.i; false if it has no work.
template <int NT>
__device__ __forceinline__ bool ck_request(const ChunkParams &p, ChunkPiece &s)
{
    const int32_t B = NT * p.R, end = __ldg(p.cu + s.i + 1);
    s.off = __ldg(p.cu + s.i);
    s.L = __ldg(p.ctx_len + s.i);
    s.k = end - s.off;
    if (s.k <= 0 || ck_bad(p, s.off, end, s.L))
        return false;
    s.nb = (s.k + B - 1) / B;
    s.wt = ck_weight<NT>(s.k, p.R);
    return true;
}

// The next pair before cost v1, from its first tile.
template <int NT>
__device__ __forceinline__ bool ck_next(const ChunkParams &p, ChunkPiece &s, int64_t v1)
{
    s.base += (int64_t)s.wt * (kStartKeys + (int64_t)s.len);
    if (s.base >= v1)
        return false;
    if (++s.b == s.nb) {
        s.b = 0;
        if (++s.g == p.c.hkv) {
            s.g = 0;
            do {
                if (++s.i >= p.n)
                    return false;     // (never: base < v1 <= the total)
            } while (!ck_request<NT>(p, s));
        }
    }
    return ck_set<NT>(p, s, v1, 0);
}

// The first piece of the share [v0, v1).
template <int NT>
__device__ __forceinline__ bool ck_first(const ChunkParams &p, const int64_t *prefix, ChunkPiece &s, int64_t v0,
                                         int64_t v1)
{
    if (v0 >= v1)
        return false;
    const int32_t B = NT * p.R;
    int32_t lo = 0, hi = p.n;
    while (hi - lo > 1) {             // last request with prefix <= v0 (it has a cost: v0 < total)
        const int32_t mid = (lo + hi) >> 1;
        if (prefix[mid] <= v0)
            lo = mid;
        else
            hi = mid;
    }
    s.i = lo;
    ck_request<NT>(p, s);
    const int32_t wt = s.wt;
    const int64_t H = ck_head_keys(s.L, s.k, B) * wt;
    int64_t rem = v0 - prefix[lo];
    s.g = (int32_t)(rem / H);
    rem -= s.g * H;
    // last block with cost before it <= rem: the root of B/2 b^2 + (a + B/2) b = rem / wt, put right
    const int64_t a = (int64_t)kStartKeys + s.L;
    const float h = (float)a + 0.5f * B;
    int64_t b = (int64_t)((sqrtf(h * h + 2.0f * B * ((float)rem / wt)) - h) / B);
    b = b < 0 ? 0 : b > s.nb - 1 ? s.nb - 1 : b;
    while (b + 1 < s.nb && ck_before(a, B, b + 1) * wt <= rem)
        ++b;
    while (b > 0 && ck_before(a, B, b) * wt > rem)
        --b;
    s.b = (int32_t)b;
    s.base = prefix[lo] + s.g * H + ck_before(a, B, b) * wt;
    const int32_t t0 = ck_tile_at(v0 - s.base, wt);
    const bool have = ck_set<NT>(p, s, v1, t0);
    // a share that begins behind the pair's last tile begins with the next pair
    return have || (t0 >= s.nt && ck_next<NT>(p, s, v1));
}

// CTA c of ncta has the costs [c, c + 1) x share; ncta shares hold the total, and a share (but the last)
// more than a tile.
struct ChunkShares {
    int64_t total, share;
    int32_t ncta;
};

__device__ __forceinline__ ChunkShares ck_shares(int64_t total)
{
    ChunkShares x;
    x.total = total;
    x.ncta = (int32_t)max((int64_t)1, min((int64_t)gridDim.x, total / kShareCost));
    x.share = max((int64_t)1, (total + x.ncta - 1) / x.ncta);
    return x;
}

// The CTA that owns the tile that starts at cost u < total.
__device__ __forceinline__ int32_t ck_owner(const ChunkShares &x, int64_t u)
{
    const int32_t c = (int32_t)(u / x.share);
    return c;
}

// Cost before each request into prefix[0..n] (shared memory that the pipeline uses later; every thread of
// the block, tot: one entry a warp).  A request that breaks the contract costs nothing, and sets a status bit.  Ends in a barrier.
template <int NT>
__device__ __forceinline__ void ck_prologue(const ChunkParams &p, int64_t *prefix, int64_t *tot)
{
    const int32_t B = NT * p.R;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nwarp = blockDim.x >> 5;
    if (tid == 0)
        prefix[0] = 0;
    int64_t running = 0;
    for (int32_t base = 0; base < p.n; base += (int32_t)blockDim.x) {
        const int32_t i = base + tid;
        int64_t cost = 0;
        if (i < p.n) {
            const int32_t off = __ldg(p.cu + i), end = __ldg(p.cu + i + 1), L = __ldg(p.ctx_len + i);
            const int32_t bad = ck_bad(p, off, end, L);
            if (bad && blockIdx.x == 0)
                set_status(p.status, bad);
            if (!bad)
                cost = ck_head_keys(L, end - off, B) * ck_weight<NT>(end - off, p.R) * p.c.hkv;
        }
        int64_t incl = cost;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o)
                incl += v;
        }
        if (lane == 31)
            tot[warp] = incl;
        __syncthreads();
        int64_t before = running;
        for (int w2 = 0; w2 < nwarp; ++w2) {
            const int64_t x = tot[w2];
            if (w2 < warp)
                before += x;
            running += x;
        }
        if (i < p.n)
            prefix[i + 1] = before + incl;
        __syncthreads();
    }
    __syncthreads();
}

__device__ __forceinline__ float ck_pow2(int32_t e)      // 2^e, e clamped to the normal range
{
    return __uint_as_float((uint32_t)(127 + max(-126, min(127, e))) << 23);
}

// Power of two that takes a query row to fp16: its largest magnitude (bf16 bits in top) to 2^14 or more, 8 bits
// of mantissa in range for elements down to 2^-31 of it.  Rows under 2^-106 are taken up by 2^120 only, so
// that the inverse times the scale is a normal number: a row of 2^-126 lies at 2^-6 and loses digits of elements
// below 2^-11 of its largest.
__device__ __forceinline__ int32_t ck_q_shift(uint32_t top)
{
    return top == 0u ? 0 : min(141 - (int32_t)(top >> 7), 120);
}

__device__ __forceinline__ uint32_t ck_pack_f16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

}  // namespace svp
