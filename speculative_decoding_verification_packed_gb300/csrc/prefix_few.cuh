// prefix_few.cuh -- svp_prefix_attn over bf16 pages: the blocks that take requests of few rows, beside those that take
// the groups (chunk_kernel.cuh, whose kernel this is a part of).
//
// Decode tokens behind a common beginning have short keys of their own, and many of them: 64 requests of 8 KV
// heads are 512 pairs of a few tiles.  The tile kernel (chunk_kernel.cuh) pays 5 us for a pair's start and end, with
// most of its 128 rows empty.  Here, as in chunk_short.cu for 8-bit pages, keys are the 16-row side of warp-level
// m16n8k16 products and query rows the 8-column side,
//   S^T (16 keys x 8 rows) = K Q^T,   O^T (16 of d x 8 rows) += V^T P^T,
// eight warps share the 128 positions of a KV tile, 16 each, and hold their rows' running maximum and sum and their
// O in registers; they join at the end of a piece through shared memory.  K and V come by TMA as the tile
// kernel's half tiles (128 rows of 64 elements, 128-byte swizzle) and are read by ldmatrix, V transposed; P^T
// turns from accumulator to operand by movmatrix.  Scores, m, l and O are fp32, P is rounded to bf16 because the
// products take 16 bits (l sums it unrounded), as in the tile kernel.
#pragma once

#include <cfloat>

#include "prefix_pieces.cuh"

namespace svp {

constexpr int kFwWarps = 8;           // computing warps; then a K and a V loader
constexpr int kFwSlots = 8;           // ring slots at most: even ones hold K, odd ones V

struct FewMisc {
    uint64_t bars[2 * kFwSlots];
    int32_t abort_flag, pad;
    float2 ml[kFwWarps][kPxRows];     // [warp][row of its request]
};

template <int D>
struct FewCfg {
    static constexpr int kSlot = (D / 64) * kCkSub;
    static constexpr int KS = D / 16;
    static constexpr int kRed = kFwWarps * kPxRows * (D + 8) * 4;   // the warps' O, rows padded
};

// C += A B, bf16 operands, fp32 accumulators (m16n8k16).
__device__ __forceinline__ void fw_mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Four 8 x 8 blocks of 16-bit elements from shared memory, row addresses by lane / 8; transposed.
__device__ __forceinline__ void fw_ld4(uint32_t addr, uint32_t (&x)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void fw_ld4t(uint32_t addr, uint32_t (&x)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                 : "r"(addr)
                 : "memory");
}

// A transposed 8 x 8 block of 16-bit pairs.
__device__ __forceinline__ uint32_t fw_turn(uint32_t x)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// 16-byte chunk c of row `row` in a slot.
__device__ __forceinline__ uint32_t fw_chunk(int row, int c)
{
    return (uint32_t)((c >> 3) * kCkSub + row * 128 + (((c & 7) ^ (row & 7)) << 4));
}

// Share [v0, v1) of the requests' costs; every thread of the block.  The joining buffer, the ring (p.few_ring, p.few_slots) and
// the barriers (p.few_misc) lie below p.off_misc, where the prologue's sums were until the first piece, s, was found.
template <int D>
__device__ __forceinline__ void few_body(const ChunkParams &p, uint8_t *smem, PrefixPiece s, bool have0, int64_t v1, int32_t cta)
{
    using Cfg = FewCfg<D>;
    constexpr int KS = Cfg::KS;
    const uint32_t sbase = smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    FewMisc *m = reinterpret_cast<FewMisc *>(smem + p.few_misc);
    const uint32_t bar0 = smem_u32(m->bars);
    auto bar_full = [&](uint32_t s) { return bar0 + 8u * s; };
    auto bar_empty = [&](uint32_t s) { return bar0 + 8u * (kFwSlots + s); };
    volatile int *abort_flag = &m->abort_flag;
    const uint32_t nslot = (uint32_t)p.few_slots;
    if (tid == 0) {
        for (int s = 0; s < kFwSlots; ++s) {
            mbar_init(bar_full(s), 1);
            mbar_init(bar_empty(s), kFwWarps);
        }
        mbar_fence_init();
        m->abort_flag = 0;
    }
    fence_proxy_async_smem();             // the loads overwrite the sums
    __syncthreads();

    if (warp == kFwWarps || warp == kFwWarps + 1) {
        // ============================================================ K loader, V loader
        // Lane u looks after positions 4 u .. 4 u + 3 of a tile; the lane of a page's first positions loads the
        // page; pages that are not needed or not in the pool are loaded from past the pool (zeros).
        const int kv = warp - kFwWarps;
        const CUtensorMap *tm = kv ? &p.tm_v : &p.tm_k;
        const uint64_t pol = l2_policy_evict_first();       // each byte is read once
        const int32_t in_page = (1 << p.c.page_shift) - 1;
        const bool loads = ((lane * 4) & in_page) == 0;
        uint32_t slot = kv, phase = 0, done = 0;
        bool ok = true;
        for (bool have = have0; have && ok; have = ck_next<1>(p, s, v1)) {
            const int32_t *bt = p.c.block_table + ck_table(p, s);
            auto needed = [&](int32_t t) { return t < s.t1 && ((t * kCkKeys + lane * 4) & ~in_page) < s.len; };
            auto page_of = [&](int32_t t) -> int32_t {
                return needed(t) ? __ldg(bt + ((t * kCkKeys + lane * 4) >> p.c.page_shift)) : -1;
            };
            int32_t id = page_of(s.t0), id1 = page_of(s.t0 + 1);
            for (int32_t t = s.t0; t < s.t1; ++t, ++done) {
                const int32_t id2 = page_of(t + 2);
                if (id < 0 || id >= p.c.num_pages) {
                    if (needed(t))
                        set_status(p.status, SVP_DEV_BAD_CONTEXT);
                    id = max(p.c.num_pages, 1);
                }
                int got = 1;
                if (lane == 0)
                    got = mbar_wait(bar_empty(slot), phase ^ 1u, abort_flag);
                if (!(ok = __shfl_sync(0xffffffffu, got, 0) != 0))
                    break;
                if (lane == 0)
                    mbar_arrive_expect_tx(bar_full(slot), (uint32_t)Cfg::kSlot);
                __syncwarp();
                if (loads) {
#pragma unroll
                    for (int c = 0; c < D / 64; ++c)
                        tma_load_4d_hint(sbase + p.few_ring + slot * Cfg::kSlot + c * kCkSub + lane * 512, tm, bar_full(slot),
                                         c * 64, 0, s.g, id, pol);
                }
                __syncwarp();
                if ((slot += 2) >= nslot) {
                    slot -= nslot;
                    phase ^= 1u;
                }
                id = id1;
                id1 = id2;
            }
        }
        if (lane == 0) {
            // every load lands before the CTA's shared memory is given back
            volatile int drain = 0;
            const uint32_t per = nslot / 2;
            for (uint32_t x = done > per ? done - per : 0u; x < done; ++x)
                mbar_wait(bar_full((2 * x + kv) % nslot), (x / per) & 1u, &drain);
        }
        __syncwarp();
    } else if (warp < kFwWarps) {
        // ============================================================ computing warps
        const int q = lane & 3, r = lane >> 2, kb = warp * 16;
        float *red = reinterpret_cast<float *>(smem);       // [8 warps][8 rows][D + 8]
        // this lane's row of the blocks that ldmatrix reads: keys kb + (0 .. 7, and + 8), chunk 0 or 1
        const int krow = kb + (lane & 15), kchunk = lane >> 4;                        // of K: blocks by key, then by d
        const int vrow = kb + (lane & 7) + (lane >> 4) * 8, vchunk = (lane >> 3) & 1; // of V: by d, then by key
        uint32_t slot = 0, phase = 0;
        bool ok = true;
        for (bool have = have0; have; have = ck_next<1>(p, s, v1)) {
            const int32_t nrows = s.ntok * p.G;
            // ---- Q: row r as operands; last visible key of rows 2 q and 2 q + 1
            uint32_t b0[KS], b1[KS];
            int32_t last[2];
            {
                const bool live = r < nrows;
                const int32_t tok = live ? r / p.G : 0, h = live ? r - tok * p.G : 0;
                const uint32_t *src = reinterpret_cast<const uint32_t *>(static_cast<const uint16_t *>(p.q) +
                                                                         (int64_t)(s.off + s.tb0 + tok) * p.q_stride +
                                                                         (int64_t)(s.g * p.G + h) * D) + q;
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    b0[k] = live ? __ldg(src + 8 * k) : 0u;
                    b1[k] = live ? __ldg(src + 8 * k + 4) : 0u;
                }
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    last[x] = 2 * q + x < nrows ? s.L + s.tb0 + (2 * q + x) / p.G : -1;
            }
            float o[KS][4], mx[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
            for (int j = 0; j < KS; ++j)
                o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.0f;
            for (int32_t t = s.t0; t < s.t1 && ok; ++t) {
                const uint32_t vs = slot + 1;               // (slots come in pairs, nslot is even)
                ok = __all_sync(0xffffffffu, mbar_wait(bar_full(slot), phase, abort_flag));
                if (!ok)
                    break;
                const int32_t k0 = t * kCkKeys + kb;        // this warp's first key
                const bool masked = k0 + 15 > s.L + s.tb0;
                const uint32_t kt = sbase + p.few_ring + slot * Cfg::kSlot, vt = sbase + p.few_ring + vs * Cfg::kSlot;
                // ---- S^T of keys k0 + r and k0 + r + 8 with rows 2 q and 2 q + 1, in two chains of products
                float sc[4], s1[4];
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    sc[x] = s1[x] = 0.0f;
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    uint32_t a[4];
                    fw_ld4(kt + fw_chunk(krow, 2 * k + kchunk), a);
                    fw_mma(k & 1 ? s1 : sc, a, b0[k], b1[k]);
                }
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    sc[x] += s1[x];
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar_empty(slot));
                // ---- the running maximum (moved when a score lies more than 2^8 above it) and P
                uint32_t pb[2];
                float top[2];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        float z = sc[2 * y + x] * p.scale_log2;
                        if (masked)
                            z = k0 + r + 8 * y <= last[x] ? z : -INFINITY;
                        sc[2 * y + x] = z;
                    }
                    top[x] = fmaxf(sc[x], sc[2 + x]);
                }
#pragma unroll
                for (int w2 = 4; w2 < 32; w2 <<= 1) {
                    top[0] = fmaxf(top[0], __shfl_xor_sync(0xffffffffu, top[0], w2));
                    top[1] = fmaxf(top[1], __shfl_xor_sync(0xffffffffu, top[1], w2));
                }
                const bool up0 = top[0] > mx[0] + kCkSlack || (mx[0] == -INFINITY && top[0] != -INFINITY);
                const bool up1 = top[1] > mx[1] + kCkSlack || (mx[1] == -INFINITY && top[1] != -INFINITY);
                if (__any_sync(0xffffffffu, up0 || up1)) {
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const float mn = fmaxf(mx[x], top[x]);
                        const float alpha = mx[x] == -INFINITY ? 0.0f : fast_exp2(mx[x] - mn);
                        mx[x] = mn;
                        l[x] *= alpha;
#pragma unroll
                        for (int j = 0; j < KS; ++j) {
                            o[j][x] *= alpha;
                            o[j][2 + x] *= alpha;
                        }
                    }
                }
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    float pr[2];
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        pr[x] = fast_exp2(sc[2 * y + x] - (mx[x] == -INFINITY ? 0.0f : mx[x]));
                        l[x] += pr[x];
                    }
                    pb[y] = fw_turn(pack_bf16x2(pr[0], pr[1]));             // row r, keys 8 y + 2 q, + 1
                }
                // ---- O^T += V^T P^T: keys k0 + 2 q, + 1 and + 8, + 9 in a thread
                ok = __all_sync(0xffffffffu, mbar_wait(bar_full(vs), phase, abort_flag));
                if (!ok)
                    break;
                // (what lies past the last visible key may be NaN, which P = 0 does not hide)
                uint32_t seen[2] = {0xffffffffu, 0xffffffffu};
                if (masked) {
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const int32_t at = k0 + 8 * y + 2 * q;
                        seen[y] = (at < s.len ? 0xffffu : 0u) | (at + 1 < s.len ? 0xffff0000u : 0u);
                    }
                }
#pragma unroll
                for (int j = 0; j < KS; ++j) {
                    uint32_t a[4];
                    fw_ld4t(vt + fw_chunk(vrow, 2 * j + vchunk), a);
                    if (masked) {
                        a[0] &= seen[0];
                        a[1] &= seen[0];
                        a[2] &= seen[1];
                        a[3] &= seen[1];
                    }
                    fw_mma(o[j], a, pb[0], pb[1]);
                }
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar_empty(vs));
                if ((slot += 2) == nslot) {
                    slot = 0;
                    phase ^= 1u;
                }
            }
            // ---- join the warps: every warp's (m, l) and O to shared memory, then four columns of a row a thread
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                float z = l[x];
#pragma unroll
                for (int w2 = 4; w2 < 32; w2 <<= 1)
                    z += __shfl_xor_sync(0xffffffffu, z, w2);
                const int row = 2 * q + x;
                if (r == 0)
                    m->ml[warp][row] = make_float2(mx[x], z);
                float *dst = red + (warp * kPxRows + row) * (D + 8) + r;
#pragma unroll
                for (int j = 0; j < KS; ++j) {
                    dst[16 * j] = o[j][x];
                    dst[16 * j + 8] = o[j][2 + x];
                }
            }
            if (named_bar_any(1, 32 * kFwWarps, !ok))
                break;                                      // (all eight warps leave together)
            const bool all = s.t0 == 0 && s.t1 == s.nt, whole = all && !ck_kept(s);
            for (int32_t idx = tid; idx < nrows * (D / 4); idx += 32 * kFwWarps) {
                const int32_t rho = idx / (D / 4), c4 = idx - rho * (D / 4);   // columns 4 c4 .. 4 c4 + 3
                float M = -INFINITY;
#pragma unroll
                for (int32_t k = 0; k < kFwWarps; ++k) {
                    const float2 x = m->ml[k][rho];
                    M = fmaxf(M, x.y != 0.0f ? x.x : -INFINITY);
                }
                float L = 0.0f, acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int32_t k = 0; k < kFwWarps; ++k) {
                    const float2 x = m->ml[k][rho];
                    if (x.y == 0.0f)
                        continue;                           // no visible key: whatever its O holds
                    const float w = fmaxf(fast_exp2(x.x - M), FLT_MIN);   // (more than 0: its O may be NaN)
                    L += w * x.y;
                    const float4 v = *reinterpret_cast<const float4 *>(red + (k * kPxRows + rho) * (D + 8) + 4 * c4);
                    acc[0] = fmaf(w, v.x, acc[0]);
                    acc[1] = fmaf(w, v.y, acc[1]);
                    acc[2] = fmaf(w, v.z, acc[2]);
                    acc[3] = fmaf(w, v.w, acc[3]);
                }
                const int32_t tok = rho / p.G, h = rho - tok * p.G;
                if (whole) {
                    const float inv = 1.0f / L;
                    const int64_t orow = (int64_t)(s.off + s.tb0 + tok) * p.hq + s.g * p.G + h;
                    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.out) + orow * D + 4 * c4) =
                        make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
                    if (c4 == 0 && p.lse)
                        p.lse[orow] = (M + __log2f(L)) * 0.69314718055994531f;
                } else {
                    int64_t prow = (int64_t)(2 * cta + (s.t0 > 0 ? 0 : 1)) * kPxRows + rho;
                    float *part_o = p.few_o;
                    float2 *part_ml = p.few_ml;
                    if (all) {
                        prow = px_place(p, false, s.off + s.tb0 + tok, s.g * p.G + h);
                        part_o = p.place_o;
                        part_ml = p.place_ml;
                    }
                    *reinterpret_cast<float4 *>(part_o + prow * D + 4 * c4) = make_float4(acc[0], acc[1], acc[2], acc[3]);
                    if (c4 == 0)
                        part_ml[prow] = make_float2(M, L);
                }
            }
            named_bar_sync(1, 32 * kFwWarps);               // the buffers are read
        }
    }
    __syncthreads();
    if (*abort_flag && tid == 0)
        set_status(p.status, SVP_DEV_TIMEOUT);
}

}  // namespace svp
