// cache.cu -- writing key / value rows into the pages of a cache, and reading them back.
//
// Write: x' = x for a cache of the rows' type; for 8-bit rows x' = rn_e4m3(x * 2^-e), e the
// smallest integer with max|x| <= 448 * 2^e over the row of one token and head.  The scale is a
// power of two on purpose: e4m3 is a floating format, so a finer scale would not save a bit of
// any element's relative precision, while a power of two makes the scaling and the way back
// exact (code * 2^e is a bf16 number) and costs one byte a row.
//
// Both kernels are bound by memory traffic once a few thousand rows are moved, and by the chain
// cu_slots -> context length -> block table -> data below that.  So a block takes a few packed
// rows of all heads: its threads look at all requests at once (one round trip) and the one
// whose request owns a row resolves the row's page; the write has its rows' data already on
// the way then, because their addresses need no lookup.  A group of d / 16 lanes moves one row
// of one head, sixteen elements a lane.
#include "svp_cache.cuh"

namespace svp {

constexpr int kCacheThreads = 128;
constexpr int kCacheRows = 4;     // packed rows of a block, at most (a read of 8-bit rows: 305 us; 16 rows 307)

struct CacheMoveParams {
    CacheParams c;
    const void *k_in, *v_in;      // write: rows
    void *k_out, *v_out;          // read: rows
    int64_t row_stride;           // elements
    const int32_t *first;         // position of each request's row 0 (ctx_len / start), or NULL
    const int32_t *cu, *take;
    int32_t n, rows, d, rpb;      // rpb: packed rows a block
    int32_t *status;
};

// Where packed row r0 + r of this block lives: slot[r] = element offset of (page, head 0, token)
// in the pools, or -1 for a row that is not moved; eoff[r] = that of its exponent byte.
struct CacheRowMap {
    int64_t slot[kCacheRows], eoff[kCacheRows];
    int32_t req[kCacheRows], pos[kCacheRows];
};

__device__ __forceinline__ void cache_locate(const CacheMoveParams &p, int32_t r0, int32_t nr, CacheRowMap &m)
{
    const int tid = threadIdx.x;
    if (tid < kCacheRows)
        m.req[tid] = -1;
    __syncthreads();
    for (int32_t i = tid; i < p.n; i += kCacheThreads) {
        const int32_t off = __ldg(p.cu + i), end = __ldg(p.cu + i + 1);
        if (off < 0 || end < off || end > p.rows) {
            if (blockIdx.x == 0)
                set_status(p.status, SVP_DEV_BAD_SLOTS);
            continue;
        }
        const int32_t lo = max(off, r0);
        int32_t hi = min(end, r0 + nr);
        if (lo >= hi)
            continue;
        const int32_t first = p.first ? __ldg(p.first + i) : 0;
        int32_t k = end - off;
        if (p.take)
            k = min(k, max(__ldg(p.take + i), 0));
        if (k == 0)
            continue;
        if (first < 0 || (int64_t)first + k > ((int64_t)p.c.max_pages << p.c.page_shift)) {
            set_status(p.status, SVP_DEV_BAD_CONTEXT);
            continue;
        }
        hi = min(hi, off + k);
        for (int32_t r = lo; r < hi; ++r) {
            m.req[r - r0] = i;
            m.pos[r - r0] = first + (r - off);
        }
    }
    __syncthreads();
    if (tid < nr) {
        const int32_t i = m.req[tid], pos = m.pos[tid];
        int64_t slot = -1, eoff = 0;
        if (i >= 0) {
            const int32_t page = __ldg(p.c.block_table + (int64_t)i * p.c.max_pages + (pos >> p.c.page_shift));
            const int32_t tok = pos & ((1 << p.c.page_shift) - 1);
            if (page >= 0 && page < p.c.num_pages) {
                slot = page * p.c.s_page + tok * p.c.s_tok;
                eoff = (((int64_t)page * p.c.hkv) << p.c.page_shift) + tok;
            } else {
                set_status(p.status, SVP_DEV_BAD_CONTEXT);
            }
        }
        m.slot[tid] = slot;
        m.eoff[tid] = eoff;
    }
    __syncthreads();
}

// The items of a block, (packed row, K or V head), in the order in which its groups of gl = d / 16 lanes
// take them; column c < hkv is K's head c, else V's c - hkv.
struct CacheItem {
    int32_t r, c;
    __device__ __forceinline__ void skip(int32_t by, int32_t cols)
    {
        c += by;
        while (c >= cols) {
            c -= cols;
            ++r;
        }
    }
};

template <int TIn, int TC>
__global__ void __launch_bounds__(kCacheThreads) cache_write_kernel(const __grid_constant__ CacheMoveParams p)
{
    __shared__ CacheRowMap m;
    griddep_launch_dependents();
    griddep_wait();
    const int32_t r0 = (int32_t)blockIdx.x * p.rpb;
    const int32_t nr = min(p.rpb, p.rows - r0), hkv = p.c.hkv, cols = 2 * hkv;
    const int gl = p.d >> 4;
    const int grp = threadIdx.x / gl, lane = threadIdx.x - grp * gl, ngrp = kCacheThreads / gl;
    // one item a group in flight: more blocks fit (with two, 159 MB of prompts took 37 us instead of 33)
    uint32_t raw[kWords<TIn>];
    CacheItem at{0, 0};
    at.skip(grp, cols);
    auto fetch = [&]() {
        if (at.r < nr) {
            const bool v = at.c >= hkv;
            load16<TIn>(v ? p.v_in : p.k_in,
                        (int64_t)(r0 + at.r) * p.row_stride + (int64_t)(v ? at.c - hkv : at.c) * p.d + lane * 16, raw);
        }
    };
    fetch();
    cache_locate(p, r0, nr, m);
    // every thread of the block runs every turn: the reduction below is over whole warps
    for (int32_t left = nr * cols; left > 0; left -= ngrp) {
        const int64_t slot = at.r < nr ? m.slot[at.r] : -1;
        const bool v = at.c >= hkv;
        const int32_t h = v ? at.c - hkv : at.c;
        const int64_t e = slot + h * p.c.s_head + lane * 16;
        void *pool = v ? p.c.v : p.c.k;
        if constexpr (TC == SVP_E4M3) {
            uint32_t amax = slot >= 0 ? amax16<TIn>(raw) : 0u;
            for (int o = gl >> 1; o > 0; o >>= 1)
                amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            if (slot >= 0) {
                const bool fine = amax < 0x7f800000u;
                const uint32_t b = fine ? exp_byte_of(amax) : 255u;
                // 2^-(b - 127): exponent field 254 - b (b >= 15, and b <= 247 for finite rows)
                const float inv = __uint_as_float((254u - b) << 23);
                uint32_t w[4] = {0u, 0u, 0u, 0u};
                if (fine) {
                    float x[16];
                    to_f32<TIn>(raw, x);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        w[i] = pack_e4m3x2(x[4 * i] * inv, x[4 * i + 1] * inv) |
                               (pack_e4m3x2(x[4 * i + 2] * inv, x[4 * i + 3] * inv) << 16);
                }
                store16<SVP_E4M3>(pool, e, w);
                if (lane == 0)
                    (v ? p.c.v_exp : p.c.k_exp)[m.eoff[at.r] + ((int64_t)h << p.c.page_shift)] = (uint8_t)b;
            }
        } else if (slot >= 0) {
            if constexpr (TIn == TC) {
                store16<TC>(pool, e, raw);                        // bits as they are
            } else {
                float x[16];
                uint32_t w[kWords<TC>];
                to_f32<TIn>(raw, x);
                from_f32<TC>(x, w);
                store16<TC>(pool, e, w);
            }
        }
        at.skip(ngrp, cols);
        fetch();
    }
}

template <int TC, int TOut>
__global__ void __launch_bounds__(kCacheThreads) cache_read_kernel(const __grid_constant__ CacheMoveParams p)
{
    constexpr int U = TC == SVP_E4M3 ? 1 : 2;   // items a group has in flight (8-bit rows: 2 took 340 us)
    __shared__ CacheRowMap m;
    griddep_launch_dependents();
    griddep_wait();
    const int32_t r0 = (int32_t)blockIdx.x * p.rpb;
    const int32_t nr = min(p.rpb, p.rows - r0), hkv = p.c.hkv, cols = 2 * hkv;
    cache_locate(p, r0, nr, m);
    const int gl = p.d >> 4;
    const int grp = threadIdx.x / gl, lane = threadIdx.x - grp * gl, ngrp = kCacheThreads / gl;
    CacheItem at{0, 0}, ahead;
    at.skip(grp, cols);
    ahead = at;
    while (at.r < nr) {
        uint32_t raw[U][kWords<TC>], b[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t slot = ahead.r < nr ? m.slot[ahead.r] : -1;
            if (slot >= 0) {
                const bool v = ahead.c >= hkv;
                const int32_t h = v ? ahead.c - hkv : ahead.c;
                load16<TC>(v ? p.c.v : p.c.k, slot + h * p.c.s_head + lane * 16, raw[u]);
                if constexpr (TC == SVP_E4M3)
                    b[u] = (v ? p.c.v_exp : p.c.k_exp)[m.eoff[ahead.r] + ((int64_t)h << p.c.page_shift)];
            }
            ahead.skip(ngrp, cols);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (at.r < nr && m.slot[at.r] >= 0) {
                const bool v = at.c >= hkv;
                const int32_t h = v ? at.c - hkv : at.c;
                const int64_t e = ((int64_t)(r0 + at.r) * hkv + h) * p.d + lane * 16;
                void *out = v ? p.v_out : p.k_out;
                if constexpr (TC == TOut) {
                    store16<TOut>(out, e, raw[u]);
                } else {
                    float x[16];
                    uint32_t w[kWords<TOut>];
                    to_f32<TC>(raw[u], x);
                    if constexpr (TC == SVP_E4M3) {
                        const float s = exp_byte_scale(b[u]);
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            x[i] *= s;
                    }
                    from_f32<TOut>(x, w);
                    store16<TOut>(out, e, w);
                }
            }
            at.skip(ngrp, cols);
        }
    }
}

int sm_count();

// Rows a block: one while that leaves fewer than four blocks an SM, then up to kCacheRows (the
// lookup is paid once a block; more rows a block did not gain once all SMs are busy).
static int32_t cache_rpb(int32_t rows)
{
    const int32_t want = rows / (4 * sm_count());
    return want < 1 ? 1 : want > kCacheRows ? kCacheRows : want;
}

template <typename F>
static svp_status cache_launch(F kernel, CacheMoveParams &p, cudaStream_t stream)
{
    p.rpb = cache_rpb(p.rows);
    const unsigned grid = (unsigned)((p.rows + p.rpb - 1) / p.rpb);
    return launch_pdl(kernel, dim3(grid), dim3(kCacheThreads), 0, stream, p) == cudaSuccess ? SVP_OK : SVP_ECUDA;
}

static bool al16(const void *q) { return (reinterpret_cast<uintptr_t>(q) & 15) == 0; }

svp_status cache_params(const svp_cache *cache, int32_t hkv, int32_t d, CacheParams &cp)
{
    if (!cache || hkv <= 0)
        return SVP_EINVAL;
    if (d != 64 && d != 128 && d != 256)
        return SVP_EUNSUPPORTED;
    const svp_dtype t = cache->dtype;
    if (t != SVP_F32 && t != SVP_BF16 && t != SVP_E4M3)
        return SVP_EUNSUPPORTED;
    if (cache->page_size != 16 && cache->page_size != 32 && cache->page_size != 64 && cache->page_size != 128)
        return SVP_EUNSUPPORTED;
    if (!cache->k || !cache->v || !cache->block_table || cache->max_pages < 0 || cache->num_pages < 0 ||
        cache->num_pages >= ((int64_t)1 << 31))
        return SVP_EINVAL;
    if ((int64_t)cache->max_pages * cache->page_size >= ((int64_t)1 << 31))
        return SVP_EUNSUPPORTED;
    if (t == SVP_E4M3 && (!cache->k_exp || !cache->v_exp || !al16(cache->k_exp) || !al16(cache->v_exp)))
        return SVP_EINVAL;
    const int64_t esz = t == SVP_F32 ? 4 : t == SVP_BF16 ? 2 : 1;
    const int64_t s[3] = {cache->stride_page, cache->stride_head, cache->stride_tok};
    for (int a = 0; a < 3; ++a)
        if (s[a] < d || (s[a] * esz) % 16 != 0)
            return SVP_EINVAL;
    if (!al16(cache->k) || !al16(cache->v))
        return SVP_EINVAL;
    cp.k = cache->k;
    cp.v = cache->v;
    cp.k_exp = cache->k_exp;
    cp.v_exp = cache->v_exp;
    cp.block_table = cache->block_table;
    cp.s_page = s[0];
    cp.s_head = s[1];
    cp.s_tok = s[2];
    cp.max_pages = cache->max_pages;
    cp.page_shift = cache->page_size == 16 ? 4 : cache->page_size == 32 ? 5 : cache->page_size == 64 ? 6 : 7;
    cp.num_pages = (int32_t)cache->num_pages;
    cp.hkv = hkv;
    return SVP_OK;
}

}  // namespace svp

using namespace svp;

extern "C" {

svp_status svp_cache_write(const void *k, const void *v, int64_t row_stride, svp_dtype dtype,
                           const svp_cache *cache, const int32_t *ctx_len, const int32_t *cu_slots,
                           const int32_t *take, int32_t n, int32_t m_cap, int32_t hkv, int32_t d,
                           void *ws, size_t ws_bytes, void *stream)
{
    if (n < 0 || m_cap < 0)
        return SVP_EINVAL;
    CacheMoveParams p{};
    const svp_status st = cache_params(cache, hkv, d, p.c);
    if (st != SVP_OK)
        return st;
    if (dtype != SVP_F32 && dtype != SVP_BF16)
        return SVP_EUNSUPPORTED;
    if (row_stride < (int64_t)hkv * d || (row_stride * (dtype == SVP_F32 ? 4 : 2)) % 16 != 0)
        return SVP_EINVAL;
    if (!ws || ws_bytes < kWsHeader)
        return SVP_EWORKSPACE;
    if (n == 0 || m_cap == 0)
        return SVP_OK;
    if (!k || !v || !ctx_len || !cu_slots || !al16(k) || !al16(v))
        return SVP_EINVAL;
    p.k_in = k;
    p.v_in = v;
    p.row_stride = row_stride;
    p.first = ctx_len;
    p.cu = cu_slots;
    p.take = take;
    p.n = n;
    p.rows = m_cap;
    p.d = d;
    p.status = static_cast<int32_t *>(ws);
    cudaStream_t s = (cudaStream_t)stream;
    if (dtype == SVP_F32) {
        switch (cache->dtype) {
        case SVP_F32: return cache_launch(cache_write_kernel<SVP_F32, SVP_F32>, p, s);
        case SVP_BF16: return cache_launch(cache_write_kernel<SVP_F32, SVP_BF16>, p, s);
        default: return cache_launch(cache_write_kernel<SVP_F32, SVP_E4M3>, p, s);
        }
    }
    switch (cache->dtype) {
    case SVP_F32: return cache_launch(cache_write_kernel<SVP_BF16, SVP_F32>, p, s);
    case SVP_BF16: return cache_launch(cache_write_kernel<SVP_BF16, SVP_BF16>, p, s);
    default: return cache_launch(cache_write_kernel<SVP_BF16, SVP_E4M3>, p, s);
    }
}

svp_status svp_cache_read(const svp_cache *cache, const int32_t *start, const int32_t *cu_rows,
                          int32_t n, int32_t rows, int32_t hkv, int32_t d, svp_dtype dtype,
                          void *k_out, void *v_out, void *ws, size_t ws_bytes, void *stream)
{
    if (n < 0 || rows < 0)
        return SVP_EINVAL;
    CacheMoveParams p{};
    const svp_status st = cache_params(cache, hkv, d, p.c);
    if (st != SVP_OK)
        return st;
    if (dtype != SVP_F32 && dtype != SVP_BF16)
        return SVP_EUNSUPPORTED;
    if (!ws || ws_bytes < kWsHeader)
        return SVP_EWORKSPACE;
    if (n == 0 || rows == 0)
        return SVP_OK;
    if (!cu_rows || !k_out || !v_out || !al16(k_out) || !al16(v_out))
        return SVP_EINVAL;
    p.k_out = k_out;
    p.v_out = v_out;
    p.first = start;
    p.cu = cu_rows;
    p.n = n;
    p.rows = rows;
    p.d = d;
    p.status = static_cast<int32_t *>(ws);
    cudaStream_t s = (cudaStream_t)stream;
    if (dtype == SVP_F32) {
        switch (cache->dtype) {
        case SVP_F32: return cache_launch(cache_read_kernel<SVP_F32, SVP_F32>, p, s);
        case SVP_BF16: return cache_launch(cache_read_kernel<SVP_BF16, SVP_F32>, p, s);
        default: return cache_launch(cache_read_kernel<SVP_E4M3, SVP_F32>, p, s);
        }
    }
    switch (cache->dtype) {
    case SVP_F32: return cache_launch(cache_read_kernel<SVP_F32, SVP_BF16>, p, s);
    case SVP_BF16: return cache_launch(cache_read_kernel<SVP_BF16, SVP_BF16>, p, s);
    default: return cache_launch(cache_read_kernel<SVP_E4M3, SVP_BF16>, p, s);
    }
}

}  // extern "C"
