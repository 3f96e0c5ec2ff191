// chunk_short.cu -- the launches of chunk_short.cuh's kernel: decode tokens and short candidate blocks over 8-bit pages.
#include <algorithm>
#include <cstring>

#include "chunk_short.cuh"

namespace svp {

template <int D, int NB>
__global__ void __launch_bounds__(kShThreads, 1) chunk_short_kernel(const __grid_constant__ ChunkParams p)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    const int tid = threadIdx.x;
    ShortMisc *m = reinterpret_cast<ShortMisc *>(smem + p.off_misc);
    if (tid == 0) {
        short_init(m);
        tma_prefetch_desc(&p.tm_k);
        tma_prefetch_desc(&p.tm_v);
    }
    griddep_launch_dependents();
    griddep_wait();
    if (tid == 0)
        p.desc[blockIdx.x].np = 0;
    int64_t *prefix = reinterpret_cast<int64_t *>(smem + p.off_ring);   // (until the loaders start)
    ck_prologue<1>(p, prefix, m->warp_tot);
    const ChunkShares shares = ck_shares(prefix[p.n]);
    const int32_t cta = blockIdx.x;
    const int64_t v0 = min(shares.total, cta * shares.share), v1 = min(shares.total, (cta + 1) * shares.share);
    ChunkPiece s;
    const bool have0 = ck_first<1>(p, prefix, s, v0, v1);
    fence_proxy_async_smem();             // the loads overwrite the sums
    __syncthreads();
    short_body<D, NB, false>(p, ShortLayout{p.off_ring, p.off_raw, p.nslot, p.part_o, p.part_ml, &p.tm_k, &p.tm_v}, m, smem, s, have0, v1, cta, shares);
}

int chunk_ctas();

template <int D, int NB>
static svp_status short_launch(ChunkParams &p, cudaStream_t stream)
{
    using Cfg = ShortCfg<D, NB>;
    constexpr int kBudget = 227 * 1024;
    const int misc = (int)(sizeof(ShortMisc) + 127) / 128 * 128;
    p.off_ring = (Cfg::kRed + 1023) / 1024 * 1024;
    p.nslot = std::min(kShSlots, (kBudget - p.off_ring - misc) / (Cfg::kRaw + 512)) / 2 * 2;
    if (p.nslot < 4)
        return SVP_EUNSUPPORTED;
    p.off_raw = p.off_ring + p.nslot * Cfg::kRaw;
    p.off_misc = p.off_raw + p.nslot * 512;
    static std::atomic<uint64_t> configured{0};
    if (set_smem_limit_once(chunk_short_kernel<D, NB>, kBudget, configured) != cudaSuccess)
        return SVP_ECUDA;
    // Back to back, 64 requests x 18000 keys (2.3 GB) take 365 us as dependents and 349 otherwise: 3 us earlier
    // do not pay from 0.4 GB on.  The host knows the block table's room only.
    const bool small = (int64_t)p.n * p.c.hkv * ((int64_t)p.c.max_pages << p.c.page_shift) * (2 * D) < ((int64_t)400 << 20);
    return launch_ctas(chunk_short_kernel<D, NB>, chunk_ctas(), kShThreads, (size_t)(p.off_misc + misc), stream, p, small,
                       false) == cudaSuccess
               ? SVP_OK
               : SVP_ECUDA;
}

svp_status chunk_short_run(ChunkParams &p, int32_t d, cudaStream_t stream)
{
    const bool one = p.G * p.R <= 8;      // rows of one block
    if (d == 64)
        return one ? short_launch<64, 1>(p, stream) : short_launch<64, 2>(p, stream);
    return one ? short_launch<128, 1>(p, stream) : short_launch<128, 2>(p, stream);
}

}  // namespace svp
