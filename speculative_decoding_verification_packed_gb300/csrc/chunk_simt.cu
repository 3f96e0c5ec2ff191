// chunk_simt.cu -- attention of new tokens over the paged cache on CUDA cores, fp32 throughout.
//
// Row j of request i (packed row cu_slots[i] + j) sees cache positions 0 .. ctx_len[i] + j:
// o = softmax(scale q K^T) V.  One CTA of 128 threads per (packed row, query head): each thread
// scores one key of a 128-key tile against the query row in shared memory, the tile's maximum
// and sum update the running softmax, and each thread accumulates d / 128 output columns.
#include "svp_cache.cuh"

namespace svp {

constexpr int kCsThreads = 128;

struct ChunkSimtParams {
    CacheParams c;
    const void *q;
    int64_t q_stride;
    const int32_t *ctx_len, *cu;
    int32_t n, m_cap, w, hq, d;
    float scale;
    void *out;
    float *lse;
    int32_t *status;
};

template <int T>
__device__ __forceinline__ float cs_elem(const void *base, int64_t e)
{
    if constexpr (T == SVP_F32)
        return __ldg(static_cast<const float *>(base) + e);
    else if constexpr (T == SVP_BF16)
        return __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t *>(base) + e) << 16);
    else {
        float f[4];
        e4m3x4_to_f32(__ldg(static_cast<const uint8_t *>(base) + e), f);
        return f[0];
    }
}

// Element offset of position t's row of head g, and its scale (8-bit rows); false: page invalid.
template <int T>
__device__ __forceinline__ bool cs_row(const ChunkSimtParams &p, int32_t i, int32_t g, int32_t t,
                                       const uint8_t *exps, int64_t &at, float &scale)
{
    const int32_t page = __ldg(p.c.block_table + (int64_t)i * p.c.max_pages + (t >> p.c.page_shift));
    if (page < 0 || page >= p.c.num_pages)
        return false;
    const int32_t tok = t & ((1 << p.c.page_shift) - 1);
    at = page * p.c.s_page + g * p.c.s_head + tok * p.c.s_tok;
    scale = 1.0f;
    if constexpr (T == SVP_E4M3)
        scale = exp_byte_scale(__ldg(exps + ((((int64_t)page * p.c.hkv + g) << p.c.page_shift) + tok)));
    return true;
}

template <int TQ, int TC>
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
        qs[e] = cs_elem<TQ>(p.q, qrow + e);
    __syncthreads();
    const int32_t nkeys = __ldg(p.ctx_len + i) + (row - __ldg(p.cu + i)) + 1;
    float m_run = -INFINITY, l_run = 0.0f;
    float acc0 = 0.0f, acc1 = 0.0f;
    for (int32_t t0 = 0; t0 < nkeys; t0 += kCsThreads) {
        const int32_t t = t0 + tid;
        float s = -INFINITY;
        if (t < nkeys) {
            int64_t at;
            float sc;
            float dot = 0.0f;
            if (cs_row<TC>(p, i, g, t, p.c.k_exp, at, sc)) {
                for (int e = 0; e < D; ++e)
                    dot = fmaf(qs[e], cs_elem<TC>(p.c.k, at + e), dot);
                dot *= sc;
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
            float sc;
            if (!cs_row<TC>(p, i, g, t0 + kk, p.c.v_exp, at, sc))
                continue;
            const float pw = ps[kk] * sc;
            if (tid < D)
                acc0 = fmaf(pw, cs_elem<TC>(p.c.v, at + tid), acc0);
            if (tid + kCsThreads < D)
                acc1 = fmaf(pw, cs_elem<TC>(p.c.v, at + tid + kCsThreads), acc1);
        }
        __syncthreads();
    }
    const float inv = 1.0f / l_run;
    auto put = [&](int32_t e, float x) {
        if constexpr (TQ == SVP_F32)
            static_cast<float *>(p.out)[orow + e] = x;
        else
            static_cast<uint16_t *>(p.out)[orow + e] = (uint16_t)(pack_bf16x2(x, 0.0f) & 0xffffu);
    };
    if (tid < D)
        put(tid, acc0 * inv);
    if (tid + kCsThreads < D)
        put(tid + kCsThreads, acc1 * inv);
    if (tid == 0 && p.lse)
        p.lse[(int64_t)row * p.hq + h] = m_run + logf(l_run);
}

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
    *bytes = kWsHeader;
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
    ChunkSimtParams p{};
    st = cache_params(cache, heads->hkv, heads->d, p.c);
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
    p.q = q;
    p.q_stride = q_row_stride;
    p.ctx_len = ctx_len;
    p.cu = cu_slots;
    p.n = n;
    p.m_cap = m_cap;
    p.w = w;
    p.hq = heads->hq;
    p.d = heads->d;
    p.scale = heads->scale != 0.0f ? heads->scale : 1.0f / sqrtf((float)heads->d);
    p.out = out;
    p.lse = lse;
    p.status = static_cast<int32_t *>(ws);
    const dim3 grid((unsigned)m_cap, (unsigned)heads->hq);
    cudaStream_t s = (cudaStream_t)stream;
    if (cache->dtype == SVP_F32)
        chunk_simt_kernel<SVP_F32, SVP_F32><<<grid, kCsThreads, 0, s>>>(p);
    else if (cache->dtype == SVP_BF16)
        chunk_simt_kernel<SVP_BF16, SVP_BF16><<<grid, kCsThreads, 0, s>>>(p);
    else
        chunk_simt_kernel<SVP_BF16, SVP_E4M3><<<grid, kCsThreads, 0, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? SVP_OK : SVP_ECUDA;
}

}  // extern "C"
