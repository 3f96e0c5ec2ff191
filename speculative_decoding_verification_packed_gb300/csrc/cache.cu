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
// the way then, because their addresses need no lookup.  A group of d / 8 lanes moves one row
// of one head, eight elements a lane (16-byte accesses for bf16).
#include "svp_cache.cuh"

namespace svp {

constexpr int kCacheThreads = 256;
constexpr int kCacheRows = 8;     // packed rows of a block, at most

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

// Eight elements of a row as fp32, from bf16 / fp32 / e4m3 storage, and back.
__device__ __forceinline__ void bf16x8_to_f32(const uint4 &w, float (&x)[8])
{
    x[0] = bf16_lo(w.x); x[1] = bf16_hi(w.x); x[2] = bf16_lo(w.y); x[3] = bf16_hi(w.y);
    x[4] = bf16_lo(w.z); x[5] = bf16_hi(w.z); x[6] = bf16_lo(w.w); x[7] = bf16_hi(w.w);
}

__device__ __forceinline__ uint4 f32_to_bf16x8(const float (&x)[8])
{
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
}

// Raw storage of eight elements of a type.
template <int T> struct Raw8;
template <> struct Raw8<SVP_F32> { float4 a, b; };
template <> struct Raw8<SVP_BF16> { uint4 a; };
template <> struct Raw8<SVP_E4M3> { uint2 a; };

template <int T>
__device__ __forceinline__ Raw8<T> raw_load(const void *base, int64_t e)
{
    Raw8<T> r;
    if constexpr (T == SVP_F32) {
        const float4 *s = reinterpret_cast<const float4 *>(static_cast<const float *>(base) + e);
        r.a = s[0];
        r.b = s[1];
    } else if constexpr (T == SVP_BF16) {
        r.a = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(base) + e);
    } else {
        r.a = *reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(base) + e);
    }
    return r;
}

template <int T>
__device__ __forceinline__ void raw_values(const Raw8<T> &r, float (&x)[8])
{
    if constexpr (T == SVP_F32) {
        x[0] = r.a.x; x[1] = r.a.y; x[2] = r.a.z; x[3] = r.a.w;
        x[4] = r.b.x; x[5] = r.b.y; x[6] = r.b.z; x[7] = r.b.w;
    } else if constexpr (T == SVP_BF16) {
        bf16x8_to_f32(r.a, x);
    } else {
        float lo[4], hi[4];
        e4m3x4_to_f32(r.a.x, lo);
        e4m3x4_to_f32(r.a.y, hi);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[e] = lo[e];
            x[4 + e] = hi[e];
        }
    }
}

template <int T>
__device__ __forceinline__ void store_values(void *base, int64_t e, const float (&x)[8])
{
    if constexpr (T == SVP_F32) {
        float4 *s = reinterpret_cast<float4 *>(static_cast<float *>(base) + e);
        s[0] = make_float4(x[0], x[1], x[2], x[3]);
        s[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        static_assert(T == SVP_BF16, "8-bit rows are stored with their exponent byte");
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(base) + e) = f32_to_bf16x8(x);
    }
}

// Items of a block: (packed row, head, K or V), one a group of gl = d / 8 lanes.
template <int TIn, int TC>
__global__ void __launch_bounds__(kCacheThreads) cache_write_kernel(const __grid_constant__ CacheMoveParams p)
{
    constexpr int U = 2;   // items a group has in flight
    __shared__ CacheRowMap m;
    griddep_launch_dependents();
    griddep_wait();
    const int32_t r0 = (int32_t)blockIdx.x * p.rpb;
    const int32_t nr = min(p.rpb, p.rows - r0);
    const int gl = p.d >> 3;
    const int grp = threadIdx.x / gl, lane = threadIdx.x - grp * gl, ngrp = kCacheThreads / gl;
    const int32_t items = nr * p.c.hkv * 2;
    Raw8<TIn> raw[U];
    auto fetch = [&](int32_t it, int u) {
        const int32_t item = it + u * ngrp;
        if (item < items) {
            const int32_t half = item & 1, rh = item >> 1, r = rh / p.c.hkv, h = rh - r * p.c.hkv;
            raw[u] = raw_load<TIn>(half ? p.v_in : p.k_in,
                                   (int64_t)(r0 + r) * p.row_stride + (int64_t)h * p.d + lane * 8);
        }
    };
#pragma unroll
    for (int u = 0; u < U; ++u)
        fetch(grp, u);
    cache_locate(p, r0, nr, m);
    // every thread of the block runs every turn: the reduction below is over whole warps
    for (int32_t it = grp; it - grp < items; it += U * ngrp) {
        if (it != grp) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                fetch(it, u);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int32_t item = it + u * ngrp;
            const bool have = item < items;
            const int32_t half = item & 1, rh = item >> 1, r = rh / p.c.hkv, h = rh - r * p.c.hkv;
            const int64_t at = have ? m.slot[r] : -1;
            const int64_t e = at + h * p.c.s_head + lane * 8;
            void *pool = half ? p.c.v : p.c.k;
            if constexpr (TC == SVP_E4M3) {
                float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                if (at >= 0)
                    raw_values<TIn>(raw[u], x);
                uint32_t amax = 0u;
#pragma unroll
                for (int v = 0; v < 8; ++v)
                    amax = max(amax, __float_as_uint(x[v]) & 0x7fffffffu);
                for (int o = gl >> 1; o > 0; o >>= 1)
                    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                if (at >= 0) {
                    const bool fine = amax < 0x7f800000u;
                    const uint32_t b = fine ? exp_byte_of(amax) : 255u;
                    // 2^-(b - 127): exponent field 254 - b (b >= 15, and b <= 247 for finite rows)
                    const float inv = fine ? __uint_as_float((254u - b) << 23) : 0.0f;
                    uint2 w = make_uint2(0u, 0u);
                    if (fine) {
                        w.x = pack_e4m3x2(x[0] * inv, x[1] * inv) | (pack_e4m3x2(x[2] * inv, x[3] * inv) << 16);
                        w.y = pack_e4m3x2(x[4] * inv, x[5] * inv) | (pack_e4m3x2(x[6] * inv, x[7] * inv) << 16);
                    }
                    *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(pool) + e) = w;
                    if (lane == 0)
                        (half ? p.c.v_exp : p.c.k_exp)[m.eoff[r] + ((int64_t)h << p.c.page_shift)] = (uint8_t)b;
                }
            } else if (at >= 0) {
                if constexpr (TIn == TC && TIn == SVP_BF16) {
                    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(pool) + e) = raw[u].a;   // bits as they are
                } else {
                    float x[8];
                    raw_values<TIn>(raw[u], x);
                    store_values<TC>(pool, e, x);
                }
            }
        }
    }
}

template <int TC, int TOut>
__global__ void __launch_bounds__(kCacheThreads) cache_read_kernel(const __grid_constant__ CacheMoveParams p)
{
    constexpr int U = 4;
    __shared__ CacheRowMap m;
    griddep_launch_dependents();
    griddep_wait();
    const int32_t r0 = (int32_t)blockIdx.x * p.rpb;
    const int32_t nr = min(p.rpb, p.rows - r0);
    cache_locate(p, r0, nr, m);
    const int gl = p.d >> 3;
    const int grp = threadIdx.x / gl, lane = threadIdx.x - grp * gl, ngrp = kCacheThreads / gl;
    const int32_t items = nr * p.c.hkv * 2;
    for (int32_t it = grp; it < items; it += U * ngrp) {
        Raw8<TC> raw[U];
        uint32_t b[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int32_t item = it + u * ngrp;
            const int32_t half = item & 1, rh = item >> 1, r = rh / p.c.hkv, h = rh - r * p.c.hkv;
            if (item < items && m.slot[r] >= 0) {
                raw[u] = raw_load<TC>(half ? p.c.v : p.c.k, m.slot[r] + h * p.c.s_head + lane * 8);
                if constexpr (TC == SVP_E4M3)
                    b[u] = (half ? p.c.v_exp : p.c.k_exp)[m.eoff[r] + ((int64_t)h << p.c.page_shift)];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int32_t item = it + u * ngrp;
            const int32_t half = item & 1, rh = item >> 1, r = rh / p.c.hkv, h = rh - r * p.c.hkv;
            if (item < items && m.slot[r] >= 0) {
                float x[8];
                raw_values<TC>(raw[u], x);
                if constexpr (TC == SVP_E4M3) {
                    const float s = exp_byte_scale(b[u]);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        x[e] *= s;
                }
                store_values<TOut>(half ? p.v_out : p.k_out, ((int64_t)(r0 + r) * p.c.hkv + h) * p.d + lane * 8, x);
            }
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
