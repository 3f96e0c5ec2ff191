// chunk_tc.cu -- svp_chunk_attn over bf16 and 8-bit pages: the launches of chunk_kernel.cuh's kernel, and the
// joining of pairs that were split between blocks.
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstring>

#include "chunk_kernel.cuh"

namespace svp {

// ------------------------------------------------------------------ joining split pairs
// Block (c, y): rows of the pair whose first piece CTA c had, one row a half warp: o = sum_q 2^(m_q - M)
// O_q / L over the pieces in their order, L = sum_q 2^(m_q - M) l_q.  Launched behind the kernel above
// as its dependent; most blocks find nothing to do.  Bound by its chain of reads, descriptor -> (m, l)
// and O: the first pieces' O are asked for together with (m, l).
constexpr int kJoinWarps = 4, kJoinRows = 2 * kJoinWarps;

template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) chunk_join_kernel(const __grid_constant__ ChunkParams p, int32_t part_rows)
{
    constexpr int E = D / 16, A = D == 256 ? 2 : 4;       // columns a lane, four side by side; pieces read ahead
    griddep_launch_dependents();
    griddep_wait();
    const int32_t c = blockIdx.x, lane = threadIdx.x & 15, half = (threadIdx.x >> 4) & 1;
    const ChunkDesc d = p.desc[c];
    const int32_t np = d.np, rows = d.ntok * p.G;
    if (np < 2)
        return;
    const float2 none = make_float2(-INFINITY, 0.0f);
    for (int32_t base = blockIdx.y * kJoinRows + (threadIdx.x >> 5) * 2; base < rows; base += kJoinRows * (int32_t)gridDim.y) {
        const int32_t rho = min(base + half, rows - 1);   // (an odd last row is done twice, and stored once)
        const int32_t tok = rho / p.G, h = rho - tok * p.G;
        const bool second = tok >= p.R;                   // token of the second query tile
        const int32_t pr = (second ? 128 : 0) + (tok - (second ? p.R : 0)) * p.G + h;
        auto at = [&](int32_t q) { return (int64_t)(q == 0 ? 2 * c + 1 : 2 * (c + q)) * part_rows + pr; };
        auto load = [&](int32_t q, float (&x)[E]) {
            const float *o = p.part_o + at(q) * D + lane * 4;
#pragma unroll
            for (int e = 0; e < E; e += 4) {
                const float4 v = __ldcg(reinterpret_cast<const float4 *>(o + 16 * e));
                x[e] = v.x;
                x[e + 1] = v.y;
                x[e + 2] = v.z;
                x[e + 3] = v.w;
            }
        };
        const float2 ml0 = lane < np ? __ldcg(p.part_ml + at(lane)) : none;
        float ahead[A][E];
#pragma unroll
        for (int q = 0; q < A; ++q)
            load(min(q, np - 1), ahead[q]);
        // (a piece without a visible key of this row, l = 0, is left out whatever its O holds)
        float M = ml0.y != 0.0f ? ml0.x : -INFINITY;
        for (int32_t q = 16 + lane; q < np; q += 16) {
            const float2 ml = __ldcg(p.part_ml + at(q));
            M = fmaxf(M, ml.y != 0.0f ? ml.x : -INFINITY);
        }
#pragma unroll
        for (int o = 8; o > 0; o >>= 1)
            M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        float acc[E], L = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e)
            acc[e] = 0.0f;
        for (int32_t q0 = 0; q0 < np; q0 += 16) {
            const float2 ml = q0 == 0 ? ml0 : q0 + lane < np ? __ldcg(p.part_ml + at(q0 + lane)) : none;
            // (more than 0 where there is a visible key: its O may be NaN)
            const float w = ml.y != 0.0f ? fmaxf(fast_exp2(ml.x - M), FLT_MIN) : 0.0f, wl = ml.y != 0.0f ? w * ml.y : 0.0f;
            auto add = [&](int32_t q, const float (&x)[E]) {
                const float wq = __shfl_sync(0xffffffffu, w, q, 16);
                L += __shfl_sync(0xffffffffu, wl, q, 16);
#pragma unroll
                for (int e = 0; e < E; ++e)
                    acc[e] = wq != 0.0f ? fmaf(wq, x[e], acc[e]) : acc[e];
            };
            int32_t q = 0;
            if (q0 == 0) {
#pragma unroll
                for (int k = 0; k < A; ++k)
                    add(k, ahead[k]);                     // (weight 0 from np on)
                q = A;
            }
            const int32_t cnt = min(16, np - q0);
#pragma unroll 2
            for (; q < cnt; ++q) {
                float x[E];
                load(q0 + q, x);
                add(q, x);
            }
        }
        if (base + half < rows) {
            const float inv = 1.0f / L;
            const int64_t orow = (int64_t)(d.row0 + tok) * p.hq + d.g * p.G + h;
            uint16_t *dst = reinterpret_cast<uint16_t *>(p.out) + orow * D + lane * 4;
#pragma unroll
            for (int e = 0; e < E; e += 4)
                *reinterpret_cast<uint2 *>(dst + 16 * e) = make_uint2(pack_bf16x2(acc[e] * inv, acc[e + 1] * inv),
                                                                      pack_bf16x2(acc[e + 2] * inv, acc[e + 3] * inv));
            if (lane == 0 && p.lse)
                p.lse[orow] = (M + __log2f(L)) * 0.69314718055994531f;
        }
        __syncwarp();
    }
}

// ------------------------------------------------------------------ host side
int sm_count();
bool encode_tiled(CUtensorMap *m, CUtensorMapDataType type, CUtensorMapSwizzle swizzle, const void *base, int rank,
                  const uint64_t *dims, const uint64_t *strides_bytes, const uint32_t *box);

int chunk_ctas() { return sm_count() & ~1; }              // (pairs)

static size_t up256(size_t x) { return (x + 255) / 256 * 256; }

struct ChunkWs {
    size_t desc, ml, o, bytes;
};

static ChunkWs chunk_ws(int32_t d)
{
    const size_t g = (size_t)chunk_ctas(), rows = d == 256 ? 128 : 256;
    ChunkWs w;
    w.desc = kWsHeader;
    w.ml = up256(w.desc + g * sizeof(ChunkDesc));
    w.o = up256(w.ml + 2 * g * rows * sizeof(float2));
    w.bytes = up256(w.o + 2 * g * rows * (size_t)d * sizeof(float));
    return w;
}

size_t chunk_tc_workspace(int32_t d) { return chunk_ws(d).bytes; }

svp_status chunk_short_run(ChunkParams &p, int32_t d, cudaStream_t stream);

template <int D>
static svp_status chunk_join(const ChunkParams &p, int32_t part_rows, cudaStream_t stream)
{
    const int rows = (int)std::min<int64_t>(part_rows, (int64_t)p.G * p.w);   // of a pair, at most
    const unsigned y = (unsigned)std::max(1, (rows + kJoinRows - 1) / kJoinRows);
    return launch_pdl(chunk_join_kernel<D>, dim3(chunk_ctas(), y), dim3(kJoinWarps * 32), 0, stream, p, part_rows) ==
                   cudaSuccess
               ? SVP_OK
               : SVP_ECUDA;
}

// Shared memory of a call whose query tiles have at most `rows` tokens: slots and offsets into p.
template <int D, bool Q8>
bool chunk_layout(ChunkParams &p, int32_t rows, int &smem)
{
    using Cfg = ChunkCfg<D, Q8>;
    constexpr int kBudget = 227 * 1024;
    // query blocks hold the rows that a piece can have; the MMA reads 128 rows whatever they are (the
    // rows behind belong to no query and their results to no output)
    p.Rb = std::min(p.R, rows);
    p.qsub = (p.G * p.Rb + 7) / 8 * 1024;
    const int qbytes = Cfg::NT * (D / 64) * p.qsub;
    const int misc = (int)(sizeof(ChunkMisc) + 127) / 128 * 128;
    p.off_ring = qbytes;
    const int room = kBudget - qbytes - misc;
    // 8-bit pages: four 16-bit slots where three raw ones fit beside them, else three
    if (Q8) {
        p.nslot = room >= 4 * Cfg::kSlot + 3 * Cfg::kRawSlot ? 4 : 3;
        p.nraw = std::min(8, (room - p.nslot * Cfg::kSlot) / Cfg::kRawSlot);
        if (p.nraw >= 2)
            p.nslot = std::min(8, (room - p.nraw * Cfg::kRawSlot) / Cfg::kSlot);
    } else {
        p.nraw = 2;
        p.nslot = std::min(8, room / Cfg::kSlot);
    }
    if (p.nslot < 3 || p.nraw < 2)
        return false;
    p.off_raw = p.off_ring + p.nslot * Cfg::kSlot;
    p.off_misc = p.off_raw + (Q8 ? p.nraw * Cfg::kRawSlot : 0);
    smem = p.off_misc + misc;
    return true;
}

template bool chunk_layout<64, false>(ChunkParams &, int32_t, int &);
template bool chunk_layout<128, false>(ChunkParams &, int32_t, int &);
template bool chunk_layout<256, false>(ChunkParams &, int32_t, int &);
template bool chunk_layout<64, true>(ChunkParams &, int32_t, int &);
template bool chunk_layout<128, true>(ChunkParams &, int32_t, int &);
template bool chunk_layout<256, true>(ChunkParams &, int32_t, int &);

template <int D, bool Q8>
static svp_status chunk_run(ChunkParams &p, cudaStream_t stream)
{
    using Cfg = ChunkCfg<D, Q8>;
    int smem = 0;
    if (!chunk_layout<D, Q8>(p, p.w, smem))
        return SVP_EUNSUPPORTED;
    static std::atomic<uint64_t> configured{0};
    if (set_smem_limit_once(chunk_tc_kernel<D, Q8, false>, 227 * 1024, configured) != cudaSuccess)
        return SVP_ECUDA;
    if (launch_ctas(chunk_tc_kernel<D, Q8, false>, chunk_ctas(), Cfg::kThreads, (size_t)smem, stream, p, true, true) !=
        cudaSuccess)
        return SVP_ECUDA;
    return chunk_join<D>(p, Cfg::kPartRows, stream);
}

// Tensor maps of the queries (boxes of box_rows tokens) and of the pages; few: for chunk_short.cu.
bool chunk_maps(ChunkParams &p, const void *q, int64_t q_stride, svp_dtype kv, int32_t m_cap, int32_t d, int32_t box_rows,
                bool few)
{
    const CacheParams &c = p.c;
    {
        const uint64_t dims[3] = {(uint64_t)d, (uint64_t)p.hq, (uint64_t)m_cap};
        const uint64_t str[2] = {(uint64_t)d * 2, (uint64_t)q_stride * 2};
        const uint32_t box[3] = {64, (uint32_t)p.G, (uint32_t)box_rows};
        if (!encode_tiled(&p.tm_q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, CU_TENSOR_MAP_SWIZZLE_128B, q, 3, dims, str, box))
            return false;
    }
    const bool q8 = kv == SVP_E4M3;
    const uint64_t esz = q8 ? 1 : 2;
    const uint64_t dims[4] = {(uint64_t)d, (uint64_t)1 << c.page_shift, (uint64_t)c.hkv,
                              (uint64_t)std::max(c.num_pages, 1)};
    const uint64_t str[3] = {(uint64_t)c.s_tok * esz, (uint64_t)c.s_head * esz, (uint64_t)c.s_page * esz};
    const uint32_t box[4] = {q8 ? (uint32_t)std::min(d, 128) : 64u, 1u << c.page_shift, 1, 1};   // a page of one head
    const CUtensorMapDataType type = q8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const CUtensorMapSwizzle sw = !q8 || (few && d == 128) ? CU_TENSOR_MAP_SWIZZLE_128B
                                  : few ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_NONE;
    return encode_tiled(&p.tm_k, type, sw, c.k, 4, dims, str, box) && encode_tiled(&p.tm_v, type, sw, c.v, 4, dims, str, box);
}

svp_status chunk_tc_launch(const void *q, int64_t q_stride, svp_dtype kv, const CacheParams &c, const int32_t *ctx_len,
                           const int32_t *cu, int32_t n, int32_t m_cap, int32_t w, int32_t hq, int32_t d, float scale,
                           void *out, float *lse, void *ws, cudaStream_t stream)
{
    ChunkParams p;
    std::memset(&p, 0, sizeof p);
    p.c = c;
    p.ctx_len = ctx_len;
    p.cu = cu;
    p.q = q;
    p.q_stride = q_stride;
    p.n = n;
    p.m_cap = m_cap;
    p.w = w;
    p.hq = hq;
    p.G = hq / c.hkv;
    p.R = 128 / p.G;
    // 8-bit pages and few rows: see chunk_short.cu
    const bool few = kv == SVP_E4M3 && d <= 128 && (int64_t)p.G * w <= kShortRows;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.out = out;
    p.out32 = (reinterpret_cast<uintptr_t>(out) & 31) == 0;
    p.lse = lse;
    const ChunkWs o = chunk_ws(d);
    uint8_t *wsb = static_cast<uint8_t *>(ws);
    p.status = reinterpret_cast<int32_t *>(wsb);
    p.desc = reinterpret_cast<ChunkDesc *>(wsb + o.desc);
    p.part_ml = reinterpret_cast<float2 *>(wsb + o.ml);
    p.part_o = reinterpret_cast<float *>(wsb + o.o);
    if (!chunk_maps(p, q, q_stride, kv, m_cap, d, std::min(p.R, w), few))
        return SVP_EUNSUPPORTED;
    if (few) {
        p.R = w;                          // a request is one token block
        const svp_status st = chunk_short_run(p, d, stream);
        if (st != SVP_OK)
            return st;
        return d == 64 ? chunk_join<64>(p, kShortRows, stream) : chunk_join<128>(p, kShortRows, stream);
    }
    if (kv == SVP_E4M3) {
        switch (d) {
        case 64: return chunk_run<64, true>(p, stream);
        case 128: return chunk_run<128, true>(p, stream);
        default: return chunk_run<256, true>(p, stream);
        }
    }
    switch (d) {
    case 64: return chunk_run<64, false>(p, stream);
    case 128: return chunk_run<128, false>(p, stream);
    default: return chunk_run<256, false>(p, stream);
    }
}

}  // namespace svp
