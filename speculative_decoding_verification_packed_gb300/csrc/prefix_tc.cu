// prefix_tc.cu -- svp_prefix_attn: chunk attention of requests in groups whose first tokens lie in the same pages.
//
// softmax over all keys of a row is the join of its softmax over the common ones and over its own:
//   M = max(m_1, m_2),  L = sum l_x 2^(m_x - M),  o = sum O_x 2^(m_x - M) / L.
// So the common keys are worked on once for all rows of a group (chunk_kernel.cuh over the sequence of
// prefix_pieces.cuh): G heads times all tokens of the group fill the 128-row tiles that a decode token alone
// leaves empty, and the pages are read once.  Every piece, of a group or of a request behind one, leaves (O, m, l)
// in fp32, the joining kernel below adds a row's pieces up in their order.  Requests alone are cut as
// svp_chunk_attn's are, but for those of few rows, which have blocks of their own beside the groups' (prefix_few.cuh).
//
// What bounds it: for few rows latency (8 tokens behind 4096, bf16: 23 us, 5.3 to the shares, 9 for a piece's chain, 5 for
// the join); else the groups' tiles (64 tokens behind 4 prefixes of 8192 to 32768, 8-bit: 109 us, 270 MB; 64 blocks of up
// to 16 rows behind 2 prefixes, bf16: 165 us, 0.65 PFLOP/s).  Where little is shared beside what the requests have
// themselves, or a decode call is small, svp_chunk_attn is quicker (2 tokens behind 256, 8192 of their own: 27 us and 25; over
// 8-bit pages 29 and 17; 8 tokens behind 4096 there 25 and 20): a group is shared by its number of blocks, not by time.
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstring>

#include "chunk_kernel.cuh"

namespace svp {

// ------------------------------------------------------------------ joining
// Where the pieces of one row's pair are: of the CTAs first .. first + np - 1, or, whole, in the row's own place.
struct PxPieces {
    int32_t first, np, pr;            // pr: the row in a CTA's partial results
};

// tok: the row among its group's, or its request's; R tokens a query tile, NT of them a block; one, two: costs of
// a key of a pair of one tile, of two.
template <int NT>
__device__ __forceinline__ PxPieces px_pieces(const ChunkParams &p, const ChunkShares &x, bool group, int64_t base, int32_t k,
                                              int32_t L, int32_t tok, int32_t g, int32_t h, int32_t R, int32_t one, int32_t two)
{
    const int32_t B = NT * R, b = tok / B, t = tok - b * B, wt = px_weight(NT, one, two, k, R);
    const int64_t H = group ? px_head_keys(L, k, B) : ck_head_keys(L, k, B);
    base += wt * (g * H + ck_before((int64_t)kStartKeys + L, group ? 0 : B, b));
    const int32_t len = group ? L : L + b * B + min(B, k - b * B), nt = (len + kCkKeys - 1) / kCkKeys;
    PxPieces y;
    y.first = ck_owner(x, base + (int64_t)wt * kStartKeys);
    y.np = ck_owner(x, base + (int64_t)wt * (kStartKeys + (int64_t)kCkKeys * (nt - 1))) - y.first + 1;
    const bool second = t >= R;
    y.pr = (second ? 128 : 0) + (t - (second ? R : 0)) * p.G + h;
    return y;
}

// Where the requests' pieces are: among the groups', or those of blocks or a kernel for few rows.
struct PxOwn {
    int32_t few, R, q8;               // tokens of its query tile; pages are 8-bit
    const float2 *ml;
    const float *o;
};

// Block (row, y): some heads of a packed row, 8 of them with a half warp each (kWays 1), or one with all eight half
// warps, which take its pieces in turn and add up through shared memory (kWays 8): calls of few rows have
// their keys cut into many pieces (8 tokens behind 4096: 20 each), which one half warp reads one after the other.
// Bound by its chain of reads, offsets -> request -> (m, l) and O.
constexpr int kPxThreads = 128, kPxHalves = kPxThreads / 16;

template <int D, int kWays>
__global__ void __launch_bounds__(kPxThreads) prefix_join_kernel(const __grid_constant__ ChunkParams p, const PxOwn w, int32_t ctas)
{
    constexpr int NT = D == 256 ? 1 : 2, kPartRows = 128 * NT;
    constexpr int E = D / 16, A = D == 256 ? 2 : 4;       // columns a lane, four side by side; pieces read ahead
    constexpr int kHeads = kPxHalves / kWays;
    __shared__ int32_t owner;
    __shared__ __align__(16) float sums[kWays > 1 ? kPxHalves : 1][D + 4];
    griddep_launch_dependents();
    griddep_wait();
    const int32_t row = blockIdx.x, tid = threadIdx.x, lane = tid & 15, way = kWays > 1 ? tid >> 4 : 0;
    if (tid == 0)
        owner = -1;
    __syncthreads();
    const int64_t total[4] = {__ldcg(p.total), __ldcg(p.total + 1), __ldcg(p.total + 2), __ldcg(p.total + 3)};
    const PxCosts cs = px_costs(p.part, total[3] != 0, w.q8 != 0);
    ChunkShares gs, os;                                   // the groups' and the requests'
    int64_t obase = 0;                                    // cost before the first request
    if (p.part == kPxBeside) {
        const int32_t split = px_split(total[0], total[1], total[2], ctas, w.q8 != 0);
        gs = ck_shares(total[1], split);
        os = ck_shares(total[0] - total[1], ctas - split);
        obase = total[1];
    } else {
        gs = os = ck_shares(total[0], ctas);
    }
    for (int32_t i = tid; i < p.n; i += kPxThreads)
        if (__ldg(p.cu + i) <= row && row < __ldg(p.cu + i + 1))
            owner = i;                                    // (one, but where nothing is computed)
    __syncthreads();
    if (owner < 0)
        return;
    const PrefixRec r = p.rec[owner];
    const PrefixGroup gr = p.grp[owner];
    const int32_t head = blockIdx.y * kHeads + (kWays > 1 ? 0 : tid >> 4);
    if (r.k <= 0 || head >= p.hq)
        return;
    const int32_t g = head / p.G, h = head - g * p.G;
    const PxPieces own = w.few ? px_pieces<1>(p, os, false, r.base - obase, r.k, r.L, row - r.off, g, h, w.R, cs.one, cs.two)
                               : px_pieces<NT>(p, os, false, r.base, r.k, r.L, row - r.off, g, h, w.R, cs.one, cs.two);
    if (r.P == 0 && own.np == 1)
        return;                                           // (the output has it already)
    PxPieces grp{0, 0, 0};
    if (r.P > 0)
        grp = px_pieces<NT>(p, gs, true, gr.base, gr.k, r.P, row - gr.off, g, h, p.R, kShortCost, cs.two);
    const int32_t np = grp.np + own.np;
    auto at = [&](int32_t q, const float2 *&ml, const float *&o) {
        const bool mine = q >= grp.np;
        const PxPieces &y = mine ? own : grp;
        q -= mine ? grp.np : 0;
        int64_t x = y.np == 1 ? px_place(p, !mine, row, head)
                              : (int64_t)(q == 0 ? 2 * y.first + 1 : 2 * (y.first + q)) * (mine && w.few ? kPxRows : kPartRows) + y.pr;
        ml = (y.np == 1 ? p.place_ml : mine ? w.ml : p.part_ml) + x;
        o = (y.np == 1 ? p.place_o : mine ? w.o : p.part_o) + x * D + lane * 4;
    };
    auto load_ml = [&](int32_t q) {
        const float2 *ml;
        const float *o;
        at(q, ml, o);
        return __ldcg(ml);
    };
    auto load = [&](int32_t q, float (&x)[E]) {
        const float2 *ml;
        const float *o;
        at(q, ml, o);
#pragma unroll
        for (int e = 0; e < E; e += 4) {
            const float4 v = __ldcg(reinterpret_cast<const float4 *>(o + 16 * e));
            x[e] = v.x;
            x[e + 1] = v.y;
            x[e + 2] = v.z;
            x[e + 3] = v.w;
        }
    };
    // (a warp's two heads may have different numbers of pieces, or one head fewer: shuffles are within the half)
    const uint32_t mask = 0xffffu << (tid & 16);
    const float2 none = make_float2(-INFINITY, 0.0f);
    const float2 ml0 = lane < np ? load_ml(lane) : none;
    float ahead[A][E];                                    // this half warp's first pieces: way, way + kWays, ..
#pragma unroll
    for (int q = 0; q < A; ++q)
        load(min(way + q * kWays, np - 1), ahead[q]);
    // (a piece without a visible key of this row, l = 0, is left out whatever its O holds)
    float M = ml0.y != 0.0f ? ml0.x : -INFINITY;
    for (int32_t q = 16 + lane; q < np; q += 16) {
        const float2 ml = load_ml(q);
        M = fmaxf(M, ml.y != 0.0f ? ml.x : -INFINITY);
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1)
        M = fmaxf(M, __shfl_xor_sync(mask, M, o, 16));
    float acc[E], L = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e)
        acc[e] = 0.0f;
    for (int32_t q0 = 0; q0 < np; q0 += 16) {
        const float2 ml = q0 == 0 ? ml0 : q0 + lane < np ? load_ml(q0 + lane) : none;
        // (more than 0 where there is a visible key: its O may be NaN)
        const float w = ml.y != 0.0f ? fmaxf(fast_exp2(ml.x - M), FLT_MIN) : 0.0f, wl = ml.y != 0.0f ? w * ml.y : 0.0f;
        auto add = [&](int32_t q, const float (&x)[E]) {  // piece q0 + q
            const float wq = __shfl_sync(mask, w, q, 16);
            L += __shfl_sync(mask, wl, q, 16);
#pragma unroll
            for (int e = 0; e < E; ++e)
                acc[e] = wq != 0.0f ? fmaf(wq, x[e], acc[e]) : acc[e];
        };
        const int32_t cnt = min(16, np - q0);
        int32_t q = way;
        if (q0 == 0) {
#pragma unroll
            for (int k = 0; k < A; ++k, q += kWays)
                if (q < 16)
                    add(q, ahead[k]);                     // (weight 0 from np on)
        } else if (q0 == 16 && kWays * A > 16) {
#pragma unroll
            for (int k = 16 / kWays; k < A; ++k, q += kWays)
                if (q < cnt)
                    add(q, ahead[k]);
        }
#pragma unroll 2
        for (; q < cnt; q += kWays) {
            float x[E];
            load(q0 + q, x);
            add(q, x);
        }
    }
    if constexpr (kWays > 1) {
#pragma unroll
        for (int e = 0; e < E; e += 4)
            *reinterpret_cast<float4 *>(&sums[way][16 * e + lane * 4]) = make_float4(acc[e], acc[e + 1], acc[e + 2], acc[e + 3]);
        if (lane == 0)
            sums[way][D] = L;
        __syncthreads();
        if (way > 0)
            return;
        for (int y = 1; y < kWays; ++y) {
            L += sums[y][D];
#pragma unroll
            for (int e = 0; e < E; e += 4) {
                const float4 v = *reinterpret_cast<const float4 *>(&sums[y][16 * e + lane * 4]);
                acc[e] += v.x;
                acc[e + 1] += v.y;
                acc[e + 2] += v.z;
                acc[e + 3] += v.w;
            }
        }
    }
    const float inv = 1.0f / L;
    const int64_t orow = (int64_t)row * p.hq + head;
    uint16_t *dst = reinterpret_cast<uint16_t *>(p.out) + orow * D + lane * 4;
#pragma unroll
    for (int e = 0; e < E; e += 4)
        *reinterpret_cast<uint2 *>(dst + 16 * e) =
            make_uint2(pack_bf16x2(acc[e] * inv, acc[e + 1] * inv), pack_bf16x2(acc[e + 2] * inv, acc[e + 3] * inv));
    if (lane == 0 && p.lse)
        p.lse[orow] = (M + __log2f(L)) * 0.69314718055994531f;
}

// ------------------------------------------------------------------ host side
int chunk_ctas();
bool chunk_maps(ChunkParams &p, const void *q, int64_t q_stride, svp_dtype kv, int32_t m_cap, int32_t d, int32_t box_rows,
                bool few);
template <int D, bool Q8>
bool chunk_layout(ChunkParams &p, int32_t rows, int &smem);

static size_t up256(size_t x) { return (x + 255) / 256 * 256; }

struct PrefixWs {
    size_t total, rec, grp, plan, ml, ml2, ml3, o, o2, o3, bytes;   // 2: of the blocks for few rows; 3: the rows' places
};

static PrefixWs prefix_ws(int32_t hq, int32_t d, int32_t m_cap)
{
    // partial results: two pieces a CTA, and those of whole pairs of groups and of requests behind them
    const size_t g = (size_t)chunk_ctas(), one = 2 * g * (d == 256 ? 128 : 256), two = 2 * g * kPxRows,
                 three = 2 * (size_t)m_cap * hq, row = (size_t)d * sizeof(float);
    PrefixWs w;
    w.total = kWsHeader;
    w.rec = w.total + 256;
    w.grp = w.rec + up256(kPxMost * sizeof(PrefixRec));
    w.plan = w.grp + up256(kPxMost * sizeof(PrefixGroup));
    w.ml = w.plan + g * 2 * kPxMost * sizeof(int4);
    w.ml2 = w.ml + up256(one * sizeof(float2));
    w.ml3 = w.ml2 + up256(two * sizeof(float2));
    w.o = w.ml3 + up256(three * sizeof(float2));
    w.o2 = w.o + one * row;
    w.o3 = w.o2 + two * row;
    w.bytes = up256(w.o3 + three * row);
    return w;
}

// Requests of at most kPxRows rows a KV head, d <= 128, have blocks of their own.
static bool few_rows(const ChunkParams &p, int32_t d) { return d <= 128 && (int64_t)p.G * p.w <= kPxRows; }

template <int D, bool Q8, bool kFew>
static svp_status prefix_tiles(const ChunkParams &p, int smem, cudaStream_t stream)
{
    static std::atomic<uint64_t> configured{0};
    if (set_smem_limit_once(chunk_tc_kernel<D, Q8, true, kFew>, 227 * 1024, configured) != cudaSuccess)
        return SVP_ECUDA;
    return launch_ctas(chunk_tc_kernel<D, Q8, true, kFew>, chunk_ctas(), ChunkCfg<D, Q8>::kThreads, (size_t)smem, stream, p, true,
                       true) == cudaSuccess
               ? SVP_OK
               : SVP_ECUDA;
}

// Shared memory of the blocks for few rows, below the tile kernel's barriers, which are moved to the end.
template <int D, bool Q8>
static bool few_layout(ChunkParams &p, int &smem)
{
    const int misc = smem - p.off_misc;
    smem = 227 * 1024;
    p.off_misc = (smem - misc) / 128 * 128;
    if constexpr (Q8) {
        using Cfg = ShortCfg<D, 1>;
        p.few_ring = (Cfg::kRed + 1023) / 1024 * 1024;
        p.few_slots = std::min(kShSlots, (p.off_misc - p.few_ring - (int)sizeof(ShortMisc)) / (Cfg::kRaw + 512)) / 2 * 2;
        p.few_raw = p.few_ring + p.few_slots * Cfg::kRaw;
        p.few_misc = p.few_raw + p.few_slots * 512;
    } else {
        using Cfg = FewCfg<D>;
        p.few_ring = (Cfg::kRed + 1023) / 1024 * 1024;
        p.few_slots = std::min(kFwSlots, (p.off_misc - p.few_ring - (int)sizeof(FewMisc)) / Cfg::kSlot) / 2 * 2;
        p.few_misc = p.few_ring + p.few_slots * Cfg::kSlot;
    }
    return p.few_slots >= 4;
}

template <int D, bool Q8>
static svp_status prefix_run(ChunkParams &p, cudaStream_t stream)
{
    using Cfg = ChunkCfg<D, Q8>;
    int smem = 0;
    p.share_rows = Cfg::NT * p.R;
    p.own_NT = Cfg::NT;
    p.own_R = p.R;
    p.part = kPxAll;
    if (!chunk_layout<D, Q8>(p, p.m_cap, smem) || p.nslot * Cfg::kSlot < (int)sizeof(PrefixSums))
        return SVP_EUNSUPPORTED;
    PxOwn own{0, p.R, Q8, p.part_ml, p.part_o};
    svp_status st;
    if (few_rows(p, D)) {
        if constexpr (D <= 128) {
            // (a pair is a request's KV head: w tokens are one block)
            p.part = kPxBeside;
            p.own_NT = 1;
            p.own_R = p.w;
            own = PxOwn{1, p.w, Q8, p.few_ml, p.few_o};
            if (!few_layout<D, Q8>(p, smem))
                return SVP_EUNSUPPORTED;
            st = prefix_tiles<D, Q8, true>(p, smem, stream);
        } else {
            return SVP_EUNSUPPORTED;                      // (never: few rows are d <= 128)
        }
    } else {
        st = prefix_tiles<D, Q8, false>(p, smem, stream);
    }
    if (st != SVP_OK)
        return st;
    const int ctas = chunk_ctas();
    // (up to four blocks an SM)
    const bool ways = (int64_t)p.m_cap * p.hq <= 4 * (int64_t)ctas;
    const dim3 grid((unsigned)p.m_cap, (unsigned)(ways ? p.hq : (p.hq + kPxHalves - 1) / kPxHalves));
    const cudaError_t e = ways ? launch_pdl(prefix_join_kernel<D, kPxHalves>, grid, dim3(kPxThreads), 0, stream, p, own, (int32_t)ctas)
                               : launch_pdl(prefix_join_kernel<D, 1>, grid, dim3(kPxThreads), 0, stream, p, own, (int32_t)ctas);
    return e == cudaSuccess ? SVP_OK : SVP_ECUDA;
}

static bool al16(const void *x) { return (reinterpret_cast<uintptr_t>(x) & 15) == 0; }
static bool al32(const void *x) { return (reinterpret_cast<uintptr_t>(x) & 31) == 0; }   // (as ck_store8 wants its parts)

}  // namespace svp

using namespace svp;

extern "C" {

svp_status svp_prefix_attn_workspace_size(const svp_heads *heads, svp_dtype dtype, int32_t m_cap, size_t *bytes)
{
    const svp_status st = svp_chunk_attn_workspace_size(heads, dtype, bytes);
    if (st != SVP_OK)
        return st;
    if (m_cap < 0)
        return SVP_EINVAL;
    if (dtype == SVP_BF16)
        *bytes = std::max(*bytes, prefix_ws(heads->hq, heads->d, m_cap).bytes);
    return SVP_OK;
}

svp_status svp_prefix_attn(const void *q, int64_t q_row_stride, const svp_cache *cache, const int32_t *ctx_len,
                           const int32_t *cu_slots, int32_t n, int32_t m_cap, int32_t w, const int32_t *cu_groups,
                           const int32_t *prefix_len, int32_t n_groups, const svp_heads *heads, svp_dtype dtype, void *out,
                           float *lse, void *ws, size_t ws_bytes, void *stream)
{
    size_t need = 0;
    svp_status st = svp_prefix_attn_workspace_size(heads, dtype, m_cap, &need);
    if (st != SVP_OK)
        return st;
    if (n_groups < 0)
        return SVP_EINVAL;
    if (n_groups > kPxMost)
        return SVP_EUNSUPPORTED;
    // no groups, fp32 pages (whose kernel reads every key for every row anyway), and every refusal
    if (n_groups == 0 || n <= 0 || n > 1024 || m_cap <= 0 || w < 1 || dtype != SVP_BF16)
        return svp_chunk_attn(q, q_row_stride, cache, ctx_len, cu_slots, n, m_cap, w, heads, dtype, out, lse, ws, ws_bytes,
                              stream);
    const float scale = heads->scale != 0.0f ? heads->scale : 1.0f / sqrtf((float)heads->d);
    if (!(scale > 0.0f) || !std::isfinite(scale))
        return SVP_EINVAL;
    ChunkParams p;
    std::memset(&p, 0, sizeof p);
    st = cache_params(cache, heads->hkv, heads->d, p.c);
    if (st != SVP_OK)
        return st;
    if (cache->dtype == SVP_F32)
        return SVP_EUNSUPPORTED;
    if (q_row_stride < (int64_t)heads->hq * heads->d || (q_row_stride * 2) % 16 != 0)
        return SVP_EINVAL;
    if (!ws || ws_bytes < need)
        return SVP_EWORKSPACE;
    if (!q || !ctx_len || !cu_slots || !cu_groups || !prefix_len || !out || !al16(q) || !al16(out) || !al32(ws))
        return SVP_EINVAL;
    const int32_t d = heads->d;
    p.ctx_len = ctx_len;
    p.cu = cu_slots;
    p.q = q;
    p.q_stride = q_row_stride;
    p.n = n;
    p.m_cap = m_cap;
    p.w = w;
    p.hq = heads->hq;
    p.G = heads->hq / heads->hkv;
    p.R = 128 / p.G;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.out = out;
    p.out32 = (reinterpret_cast<uintptr_t>(out) & 31) == 0;
    p.lse = lse;
    p.cu_groups = cu_groups;
    p.prefix_len = prefix_len;
    p.ng = n_groups;
    const PrefixWs o = prefix_ws(p.hq, d, m_cap);
    uint8_t *b = static_cast<uint8_t *>(ws);
    p.status = reinterpret_cast<int32_t *>(b);
    p.total = reinterpret_cast<int64_t *>(b + o.total);
    p.rec = reinterpret_cast<PrefixRec *>(b + o.rec);
    p.grp = reinterpret_cast<PrefixGroup *>(b + o.grp);
    p.plan = reinterpret_cast<int4 *>(b + o.plan);
    p.part_ml = reinterpret_cast<float2 *>(b + o.ml);
    p.part_o = reinterpret_cast<float *>(b + o.o);
    p.place_ml = reinterpret_cast<float2 *>(b + o.ml3);
    p.place_o = reinterpret_cast<float *>(b + o.o3);
    if (!chunk_maps(p, q, q_row_stride, cache->dtype, m_cap, d, std::min(p.R, m_cap), false))
        return SVP_EUNSUPPORTED;
    p.few_ml = reinterpret_cast<float2 *>(b + o.ml2);
    p.few_o = reinterpret_cast<float *>(b + o.o2);
    if (cache->dtype == SVP_E4M3 && few_rows(p, d)) {
        // (the pages once more, with the swizzle of chunk_short.cuh)
        ChunkParams few = p;
        if (!chunk_maps(few, q, q_row_stride, cache->dtype, m_cap, d, 1, true))
            return SVP_EUNSUPPORTED;
        p.few_k = few.tm_k;
        p.few_v = few.tm_v;
    }
    cudaStream_t s = (cudaStream_t)stream;
    if (cache->dtype == SVP_E4M3) {
        switch (d) {
        case 64: return prefix_run<64, true>(p, s);
        case 128: return prefix_run<128, true>(p, s);
        default: return prefix_run<256, true>(p, s);
        }
    }
    switch (d) {
    case 64: return prefix_run<64, false>(p, s);
    case 128: return prefix_run<128, false>(p, s);
    default: return prefix_run<256, false>(p, s);
    }
}

}  // extern "C"
