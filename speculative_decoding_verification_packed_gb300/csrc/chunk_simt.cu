// chunk_simt.cu -- svp_chunk_attn's checks, and its fp32 form on CUDA cores (fp32 throughout; tf32
// tensor cores would round the scores to 11 bits).  bf16 queries go to chunk_tc.cu.
//
// Row j of request i (packed row cu_slots[i] + j) sees cache positions 0 .. ctx_len[i] + j:
// o = softmax(scale q K^T) V.  One CTA of 128 threads per (packed row, query head): each thread
// scores one key of a 128-key tile against the query row in shared memory, the tile's maximum
// and sum update the running softmax, and each thread accumulates d / 128 output columns.
#include <cmath>

#include "svp_cache.cuh"

namespace svp {

constexpr int kCsThreads = 128;

struct ChunkSimtParams {
    CacheParams c;
    const float *q;
    int64_t q_stride;
    const int32_t *ctx_len, *cu;
    int32_t n, m_cap, w, hq, d;
    float scale;
    float *out, *lse;
    int32_t *status;
};

// Element offset of position t's row of head g; false: the page is invalid.
__device__ __forceinline__ bool cs_row(const ChunkSimtParams &p, int32_t i, int32_t g, int32_t t, int64_t &at)
{
    const int32_t page = __ldg(p.c.block_table + (int64_t)i * p.c.max_pages + (t >> p.c.page_shift));
    if (page < 0 || page >= p.c.num_pages)
        return false;
    at = page * p.c.s_page + g * p.c.s_head + (t & ((1 << p.c.page_shift) - 1)) * p.c.s_tok;
    return true;
}

__global__ void __launch_bounds__(kCsThreads) chunk_simt_kernel(const __grid_constant__ ChunkSimtParams p)
{
    __shared__ float qs[256];
    __shared__ float ps[kCsThreads];
    __shared__ float red[kCsThreads / 32];
    __shared__ int32_t owner;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t row = blockIdx.x, h = blockIdx.y;
    if (tid == 0)
        owner = -1;
    __syncthreads();
    for (int32_t i = tid; i < p.n; i += kCsThreads) {
        const int32_t off = __ldg(p.cu + i), end = __ldg(p.cu + i + 1);
        if (off < 0 || end < off || end - off > p.w || end > p.m_cap) {
            if (row == 0 && h == 0)
                set_status(p.status, SVP_DEV_BAD_SLOTS);
            continue;
        }
        if (off <= row && row < end) {
            const int32_t L = __ldg(p.ctx_len + i);
            if (L < 0 || (int64_t)L + (end - off) > ((int64_t)p.c.max_pages << p.c.page_shift))
                set_status(p.status, SVP_DEV_BAD_CONTEXT);
            else
                owner = i;
        }
    }
    __syncthreads();
    const int32_t i = owner;
    if (i < 0)
        return;
    const int32_t D = p.d, G = p.hq / p.c.hkv, g = h / G;
    const int64_t qrow = (int64_t)row * p.q_stride + (int64_t)h * D;
    const int64_t orow = ((int64_t)row * p.hq + h) * D;
    for (int e = tid; e < D; e += kCsThreads)
        qs[e] = __ldg(p.q + qrow + e);
    __syncthreads();
    const int32_t nkeys = __ldg(p.ctx_len + i) + (row - __ldg(p.cu + i)) + 1;
    float m_run = -INFINITY, l_run = 0.0f;
    float acc0 = 0.0f, acc1 = 0.0f;
    for (int32_t t0 = 0; t0 < nkeys; t0 += kCsThreads) {
        const int32_t t = t0 + tid;
        float s = -INFINITY;
        if (t < nkeys) {
            int64_t at;
            float dot = 0.0f;
            if (cs_row(p, i, g, t, at)) {
                const float *kr = static_cast<const float *>(p.c.k) + at;
                for (int e = 0; e < D; ++e)
                    dot = fmaf(qs[e], __ldg(kr + e), dot);
            } else {
                set_status(p.status, SVP_DEV_BAD_CONTEXT);   // a page of zeros
            }
            s = dot * p.scale;
        }
        float mt = s;
        for (int o = 16; o > 0; o >>= 1)
            mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
        if (lane == 0)
            red[warp] = mt;
        __syncthreads();
        mt = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
        __syncthreads();
        const float m_new = fmaxf(m_run, mt);
        // (a maximum of -inf, every score so far -inf or NaN, leaves the exponents NaN as the formula does)
        const float alpha = (m_run == -INFINITY) ? 0.0f : expf(m_run - m_new);
        const float pk = t < nkeys ? expf(s - m_new) : 0.0f;
        ps[tid] = pk;
        float sum = pk;
        for (int o = 16; o > 0; o >>= 1)
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0)
            red[warp] = sum;
        __syncthreads();
        l_run = l_run * alpha + ((red[0] + red[1]) + (red[2] + red[3]));
        m_run = m_new;
        acc0 *= alpha;
        acc1 *= alpha;
        const int32_t cnt = min(kCsThreads, nkeys - t0);
        for (int32_t kk = 0; kk < cnt; ++kk) {
            int64_t at;
            if (!cs_row(p, i, g, t0 + kk, at))
                continue;
            const float pw = ps[kk];
            const float *vr = static_cast<const float *>(p.c.v) + at;
            if (tid < D)
                acc0 = fmaf(pw, __ldg(vr + tid), acc0);
            if (tid + kCsThreads < D)
                acc1 = fmaf(pw, __ldg(vr + tid + kCsThreads), acc1);
        }
        __syncthreads();
    }
    const float inv = 1.0f / l_run;
    if (tid < D)
        p.out[orow + tid] = acc0 * inv;
    if (tid + kCsThreads < D)
        p.out[orow + tid + kCsThreads] = acc1 * inv;
    if (tid == 0 && p.lse)
        p.lse[(int64_t)row * p.hq + h] = m_run + logf(l_run);
}

size_t chunk_tc_workspace(int32_t d);
svp_status chunk_tc_launch(const void *q, int64_t q_stride, svp_dtype kv, const CacheParams &c, const int32_t *ctx_len,
                           const int32_t *cu, int32_t n, int32_t m_cap, int32_t w, int32_t hq, int32_t d, float scale,
                           void *out, float *lse, void *ws, cudaStream_t stream);

static bool al16(const void *q) { return (reinterpret_cast<uintptr_t>(q) & 15) == 0; }

}  // namespace svp

using namespace svp;

extern "C" {

svp_status svp_chunk_attn_workspace_size(const svp_heads *heads, svp_dtype dtype, size_t *bytes)
{
    if (!heads || !bytes || heads->hq <= 0 || heads->hkv <= 0 || heads->hq % heads->hkv)
        return SVP_EINVAL;
    if (heads->d != 64 && heads->d != 128 && heads->d != 256)
        return SVP_EUNSUPPORTED;
    if ((dtype != SVP_F32 && dtype != SVP_BF16) || heads->hq / heads->hkv > 128)
        return SVP_EUNSUPPORTED;
    *bytes = dtype == SVP_F32 ? kWsHeader : chunk_tc_workspace(heads->d);
    return SVP_OK;
}

svp_status svp_chunk_attn(const void *q, int64_t q_row_stride, const svp_cache *cache,
                          const int32_t *ctx_len, const int32_t *cu_slots, int32_t n,
                          int32_t m_cap, int32_t w, const svp_heads *heads, svp_dtype dtype,
                          void *out, float *lse, void *ws, size_t ws_bytes, void *stream)
{
    size_t need = 0;
    svp_status st = svp_chunk_attn_workspace_size(heads, dtype, &need);
    if (st != SVP_OK)
        return st;
    if (n < 0 || m_cap < 0 || w < 1)
        return SVP_EINVAL;
    if (n > 1024)
        return SVP_EUNSUPPORTED;
    const float scale = heads->scale != 0.0f ? heads->scale : 1.0f / sqrtf((float)heads->d);
    if (!(scale > 0.0f) || !std::isfinite(scale))
        return SVP_EINVAL;
    CacheParams c{};
    st = cache_params(cache, heads->hkv, heads->d, c);
    if (st != SVP_OK)
        return st;
    if ((dtype == SVP_F32) != (cache->dtype == SVP_F32))
        return SVP_EUNSUPPORTED;
    if (q_row_stride < (int64_t)heads->hq * heads->d || (q_row_stride * (dtype == SVP_F32 ? 4 : 2)) % 16 != 0)
        return SVP_EINVAL;
    if (!ws || ws_bytes < need)
        return SVP_EWORKSPACE;
    if (n == 0 || m_cap == 0)
        return SVP_OK;
    if (!q || !ctx_len || !cu_slots || !out || !al16(q) || !al16(out))
        return SVP_EINVAL;
    if (dtype == SVP_BF16)
        return chunk_tc_launch(q, q_row_stride, cache->dtype, c, ctx_len, cu_slots, n, m_cap, w, heads->hq, heads->d,
                               scale, out, lse, ws, (cudaStream_t)stream);
    ChunkSimtParams p{};
    p.c = c;
    p.q = static_cast<const float *>(q);
    p.q_stride = q_row_stride;
    p.ctx_len = ctx_len;
    p.cu = cu_slots;
    p.n = n;
    p.m_cap = m_cap;
    p.w = w;
    p.hq = heads->hq;
    p.d = heads->d;
    p.scale = scale;
    p.out = static_cast<float *>(out);
    p.lse = lse;
    p.status = static_cast<int32_t *>(ws);
    chunk_simt_kernel<<<dim3((unsigned)m_cap, (unsigned)heads->hq), kCsThreads, 0, (cudaStream_t)stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? SVP_OK : SVP_ECUDA;
}

}  // extern "C"
