// chunk_kernel.cuh -- attention of new tokens over the paged cache on tcgen05, bf16 and 8-bit pages: the kernel of
// chunk_tc.cu and, with kShared (groups of requests whose first tokens lie in the same pages), of prefix_tc.cu.
//
// Row j of request i sees cache positions 0 .. ctx_len[i] + j: o = softmax(scale q K^T) V.
//
// Tiles.  The G query heads that share a KV head are packed with R = 128 / G tokens into a
// 128-row query tile (row = token * G + head), so a key / value tile of 128 positions serves
// all of them:  S = Q K^T (TMEM, 128 x 128 fp32), P = 2^(S c - m) in 16 bits over the first
// half of S's columns, O += P V with P taken straight from TMEM.  One thread owns one row.
//   * long pieces (more than R tokens, d <= 128): two query tiles share one K / V stream; the
//     softmax of one runs while the tensor pipe works on the other.
//   * short pieces (decode tokens, candidate blocks): one query tile, and the two softmax
//     warpgroups take alternate KV tiles with an accumulator and a running (m, l) each; the
//     first joins them in TMEM at the end.
//   * d = 256: O fills the TMEM that a second tile would need, so one warpgroup works through
//     one query tile with two S buffers (its MMAs take twice as long a tile).
// The exponent reference m is the row's maximum over the piece's first tile; it moves (and O is
// rescaled) only when a later score lies more than 2^8 above it; over bf16 pages a full tile is first tried
// with the reference as it is, and only looked through where a row's sum exceeds 2^15.  Scores, m, l and O are fp32; P is
// rounded to bf16 because the products take 16 bits (l sums it unrounded), the output to its type.
//
// Warps.  Two loaders take the ring's positions in turn (one, alone, is bound by issuing the copies of
// 16-token pages: 64 requests x 8 rows over 8-bit pages took 808 us, two 634), two warps issue
// MMAs, the softmax has four warps a query tile, and 8-bit pages four more.
//
// 8-bit rows.  Those four warps turn the raw tile (e4m3 codes by TMA, the rows' exponents beside them
// as fp16 multipliers) into the fp16 tile that the MMAs read, in units of the tile's largest power of
// two 2^E.  A code has 4 bits of mantissa and fp16 11 and 2^-24 as its smallest step, so elements are
// exact down to 2^-15 of the tile's largest row scale, and what lies under 2^-25 of it becomes zero.
// K's E multiplies the softmax factor; V's goes into the exponent, P' = 2^(s c + E - m) with m the
// running maximum of s c + E, so tiles of any E add up in one accumulator; l takes E back out.  The
// query is made fp16 in shared memory, each row times the power of two that leaves it 15 bits of range.
// fp16 rather than bf16: P' is rounded 8 times finer, and a code widens in one conversion.  What fp16 lacks
// in range is made up by the units (above) and by P' = 2^7 at the reference.
//
// What bounds it.  Short pieces over bf16 pages: their bytes (64 requests x 18000 keys, 8 KV heads, d 128:
// 674 us, 7.0 TB/s; with 8 rows each 676 us).  Over 8-bit pages: the chains of the two warpgroups, 2.7 us a tile each,
// with the conversion, and the shared memory that it shares with the MMAs, beside them (8 rows each 649 us for half the
// bytes; 639 with 128-token pages, and 570 at d 64, with half the conversion).  Prompts: the chain S -> softmax -> P V of a
// tile (4096 rows on 8192 keys, 32 heads: 496 to 519 us by the data, 1.32 to 1.39 PFLOP/s, 8-bit pages 641; the
// MMAs alone 342 us; the exponentials keep their pipe busy for 29 % of it, all instructions the issue slots
// for 32 %).
//
// Split.  Work is the sequence of pairs (request, KV head, token block); a pair costs its
// keys plus kStartKeys, and every CTA (one per SM) takes an equal share of the total, so long
// prompts, blocks and single tokens balance in one launch.  All bounds follow in closed form
// from per-request prefix sums; the first and last piece of a CTA may be parts of a pair, whose
// (O, m, l) go to the workspace and are joined by a second kernel in the pieces' order.
#pragma once

#include <cfloat>
#include <type_traits>

#include "chunk_short.cuh"
#include "prefix_few.cuh"

namespace svp {

template <int D, bool Q8>
struct ChunkCfg {
    static constexpr int NT = D == 256 ? 1 : 2;            // query tiles of a long piece
    static constexpr int NH = D == 256 ? 2 : 1;            // 128-column halves of d
    static constexpr int DH = D / NH;
    static constexpr int kSlot = (DH / 64) * kCkSub;       // a half tile in 16 bits
    static constexpr int kRaw = kCkKeys * DH;              // and in codes
    static constexpr int kRawSlot = kRaw + 2 * kCkKeys;    // + the rows' multipliers
    // warps: 0 and 3 loaders, 1 and 2 MMA issuers, then warpgroups of softmax and converting warps
    static constexpr int kSoftWarp0 = 4;
    static constexpr int kConvWarp0 = kSoftWarp0 + 4 * NT;
    static constexpr int kConvWarps = Q8 ? 4 : 0;
    static constexpr bool kByKind = NH == 1;               // the loaders share a ring by K and V, else by halves of d
    static constexpr int kThreads = 32 * (kConvWarp0 + kConvWarps);
    static constexpr int kPartRows = 128 * NT;
};

struct ChunkMisc {
    uint64_t bars[54];
    uint32_t tmem;
    int32_t abort_flag;
    int64_t warp_tot[20];
    float2 ml[128];                   // (m, l) of the second warpgroup's half of a short piece
    float o_scale;                    // and what its O is to be multiplied with
    float2 scales[16];                // 8-bit pages: (2^E of K, E of V) of a KV tile, by tile mod 16
};

// ------------------------------------------------------------------ small device helpers
// D[tmem] (+)= A[tmem] * B[smem], bf16 or fp16 inputs, fp32 accumulate.
__device__ __forceinline__ void ck_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void ck_st_v2(uint32_t addr, uint32_t a, uint32_t b)
{
    asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}

// True in one lane of a converged warp, always the same.
__device__ __forceinline__ bool ck_elect()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

// Four codes to fp16, times the row's power of two (both halves of mul).
__device__ __forceinline__ void ck_codes(uint32_t w, uint32_t mul, uint32_t &lo, uint32_t &hi)
{
    asm("{\n\t.reg .b16 a, b;\n\t.reg .b32 x, y;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 x, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 y, b;\n\t"
        "mul.rn.f16x2 %0, x, %3;\n\t"
        "mul.rn.f16x2 %1, y, %3;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w), "r"(mul));
}

// The softmax of one S tile in this thread's row, 64 columns a turn: its instructions are kept few, as
// seven kinds of warps share the instruction cache (both passes unrolled over whole rows took twice as long).

// 32 columns of this thread's TMEM lane, and the largest of them.
__device__ __forceinline__ float ck_ld32_max(uint32_t taddr, uint32_t (&r)[32])
{
    float mx;
    asm volatile(
        "tcgen05.ld.red.sync.aligned.32x32b.x32.max.f32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, %32, [%33];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
          "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
          "=r"(r[31]), "=f"(mx)
        : "r"(taddr));
    return mx;
}

// Largest raw score; with kMasked, keys past kmax are hidden.
template <bool kMasked>
__device__ __forceinline__ float ck_row_max(uint32_t ts, int32_t kmax)
{
    float mx = -INFINITY;
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
        uint32_t sa[32], sb[32];
        const float ma = ck_ld32_max(ts + half * 64, sa), mb = ck_ld32_max(ts + half * 64 + 32, sb);
        tmem_wait_ld();
        if (!kMasked) {
            mx = fmaxf(mx, fmaxf(ma, mb));
        } else {
            const int32_t left = kmax - half * 64;
#pragma unroll
            for (int e = 0; e < 32; ++e) {
                mx = fmaxf(mx, e <= left ? __uint_as_float(sa[e]) : -INFINITY);
                mx = fmaxf(mx, e + 32 <= left ? __uint_as_float(sb[e]) : -INFINITY);
            }
        }
    }
    return mx;
}

// P = 2^(s * cl2 - m) in 16 bits over the first half of S's columns (a turn's P lies over scores that it or
// an earlier turn has read); returns its sum in fp32.
template <bool kMasked, bool F16>
__device__ __forceinline__ float ck_row_exp(uint32_t ts, int32_t kmax, float cl2, float m)
{
    const uint64_t c2 = f32x2_pack(cl2, cl2), nm2 = f32x2_pack(-m, -m);
    uint64_t acc[2] = {f32x2_pack(0.0f, 0.0f), f32x2_pack(0.0f, 0.0f)};
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
        uint32_t sv[2][32], pk[32];
        tmem_ld32(ts + half * 64, sv[0]);
        tmem_ld32(ts + half * 64 + 32, sv[1]);
        tmem_wait_ld();
        const int32_t left = kmax - half * 64;
#pragma unroll
        for (int e = 0; e < 32; ++e) {
            const int k0 = 2 * e;
            float s0 = __uint_as_float(sv[k0 >> 5][k0 & 31]);
            float s1 = __uint_as_float(sv[k0 >> 5][(k0 & 31) + 1]);
            if (kMasked) {
                s0 = k0 <= left ? s0 : -INFINITY;
                s1 = k0 + 1 <= left ? s1 : -INFINITY;
            }
            float y0, y1;
            f32x2_unpack(f32x2_fma(f32x2_pack(s0, s1), c2, nm2), y0, y1);
            const float p0 = fast_exp2(y0), p1 = fast_exp2(y1);
            pk[e] = F16 ? ck_pack_f16x2(p0, p1) : pack_bf16x2(p0, p1);
            acc[e & 1] = f32x2_add(acc[e & 1], f32x2_pack(p0, p1));
        }
        tmem_st32(ts + half * 32, pk);
    }
    float s[4];
    f32x2_unpack(acc[0], s[0], s[1]);
    f32x2_unpack(acc[1], s[2], s[3]);
    return (s[0] + s[1]) + (s[2] + s[3]);
}

// The same of an unmasked tile in one reading, with a reference from before: if every live row's sum stays
// within limit (it does not with no reference, -inf, nor with NaN), P is stored, else nothing is and the
// scores are still there.
template <bool F16>
__device__ __forceinline__ bool ck_row_once(uint32_t ts, float cl2, float m, float limit, bool live, float &sum)
{
    const uint64_t c2 = f32x2_pack(cl2, cl2), nm2 = f32x2_pack(-m, -m);
    uint64_t acc[2] = {f32x2_pack(0.0f, 0.0f), f32x2_pack(0.0f, 0.0f)};
    uint32_t p0[32], p1[32];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        uint32_t sv[2][32];
        tmem_ld32(ts + half * 64, sv[0]);
        tmem_ld32(ts + half * 64 + 32, sv[1]);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e) {
            const int k0 = 2 * e;
            float y0, y1;
            f32x2_unpack(f32x2_fma(f32x2_pack(__uint_as_float(sv[k0 >> 5][k0 & 31]),
                                              __uint_as_float(sv[k0 >> 5][(k0 & 31) + 1])), c2, nm2), y0, y1);
            y0 = fast_exp2(y0);
            y1 = fast_exp2(y1);
            (half ? p1 : p0)[e] = F16 ? ck_pack_f16x2(y0, y1) : pack_bf16x2(y0, y1);
            acc[e & 1] = f32x2_add(acc[e & 1], f32x2_pack(y0, y1));
        }
    }
    float s[4];
    f32x2_unpack(acc[0], s[0], s[1]);
    f32x2_unpack(acc[1], s[2], s[3]);
    sum = (s[0] + s[1]) + (s[2] + s[3]);
    if (!__all_sync(0xffffffffu, !live || sum <= limit))
        return false;
    tmem_st32(ts, p0);
    tmem_st32(ts + 32, p1);
    return true;
}

// 32 bytes, a whole sector, in one store (16-byte ones of a row leave half sectors).
__device__ __forceinline__ void ck_store8(void *at, const uint32_t *x)
{
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(at), "r"(x[0]), "r"(x[1]), "r"(x[2]),
                 "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                 : "memory");
}

// ------------------------------------------------------------------ the kernel
// kFew: the requests, of few rows, have blocks of their own (kPxBeside).
template <int D, bool Q8, bool kShared, bool kFew = false>
__global__ void __launch_bounds__(ChunkCfg<D, Q8>::kThreads, 1) chunk_tc_kernel(const __grid_constant__ ChunkParams p)
{
    using Cfg = ChunkCfg<D, Q8>;
    using Piece = std::conditional_t<kShared, PrefixPiece, ChunkPiece>;
    constexpr int NT = Cfg::NT, NH = Cfg::NH, DH = Cfg::DH;
    constexpr bool kMono = NT == 1;
    constexpr int kGiveAt = DH / 16 * 3 / 4;   // (products of S before the turn is given: 6 of 8 beat 4 and 2)
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    ChunkMisc *m = reinterpret_cast<ChunkMisc *>(smem + p.off_misc);
    const uint32_t bar0 = smem_u32(m->bars);
    // 16-bit tile slots (filled by TMA, or by the converting warps), raw slots
    auto bar_full = [&](int s) { return bar0 + 8u * s; };
    auto bar_empty = [&](int s) { return bar0 + 8u * (8 + s); };
    auto bar_rfull = [&](int s) { return bar0 + 8u * (16 + s); };
    auto bar_rempty = [&](int s) { return bar0 + 8u * (24 + s); };
    auto bar_q = [&](int a) { return bar0 + 8u * (32 + a); };        // query tile a is loaded
    auto bar_s = [&](int a) { return bar0 + 8u * (34 + a); };        // S buffer a is complete
    auto bar_p = [&](int a) { return bar0 + 8u * (36 + a); };        // P buffer a is written
    auto bar_o = [&](int a) { return bar0 + 8u * (38 + a); };        // O_a of the piece is complete
    auto bar_ofree = [&](int a) { return bar0 + 8u * (40 + a); };    // and has been read
    auto bar_pv = [&](int a) { return bar0 + 8u * (42 + a); };       // d = 256: P buffer a has been read
    const uint32_t bar_ml = bar0 + 8u * 44, bar_mlfree = bar0 + 8u * 45;
    auto bar_drain = [&](int a) { return bar0 + 8u * (46 + a); };
    const uint32_t bar_sdone = bar0 + 8u * 48;                       // d = 256: every S of a piece is done
    auto bar_turn = [&](int a) { return bar0 + 8u * (49 + a); };     // long pieces: issuer a's turn
    auto bar_qc = [&](int a) { return bar0 + 8u * (51 + a); };       // 8-bit pages: query tile a is in fp16
    volatile int *abort_flag = &m->abort_flag;
    const int32_t nslot = p.nslot, nraw = p.nraw;

    if (tid == 0) {
        for (int s = 0; s < 8; ++s) {
            mbar_init(bar_full(s), Q8 ? Cfg::kConvWarps : 1);
            mbar_init(bar_empty(s), 2);                              // one release from each issuer
            mbar_init(bar_rfull(s), 1);
            mbar_init(bar_rempty(s), Q8 ? Cfg::kConvWarps : 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(bar_q(a), 1);
            mbar_init(bar_turn(a), 1);
            mbar_init(bar_qc(a), 4);
            mbar_init(bar_pv(a), 1);
            mbar_init(bar_drain(a), 1);
            mbar_init(bar_s(a), 1);
            mbar_init(bar_p(a), 4);
            mbar_init(bar_o(a), 1);
            mbar_init(bar_ofree(a), 4);
        }
        mbar_init(bar_ml, 4);
        mbar_init(bar_mlfree, 4);
        mbar_init(bar_sdone, 1);
        mbar_fence_init();
        m->abort_flag = 0;
        tma_prefetch_desc(&p.tm_q);
        tma_prefetch_desc(&p.tm_k);
        tma_prefetch_desc(&p.tm_v);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&m->tmem), 512);
        tmem_relinquish();
    }
    griddep_launch_dependents();
    griddep_wait();
    if (!kShared && tid == 0)
        p.desc[blockIdx.x].np = 0;
    // costs before each request, or group and request (until the loaders start)
    using Sums = std::conditional_t<kShared, PrefixSums, int64_t[1]>;
    Sums &sums = *reinterpret_cast<Sums *>(smem + p.off_ring);
    int32_t pairs = p.n;
    if constexpr (kShared)
        pairs = px_prologue<NT>(p, smem + p.off_ring, kFew ? kPxBeside : kPxAll, Q8);
    else
        ck_prologue<NT>(p, sums, m->warp_tot);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = m->tmem;
    // kFew: of this block's kind, the groups' (the first blocks) or the requests'
    const int32_t split = [&]() -> int32_t {
        if constexpr (kFew)
            return px_split(px_total(sums, pairs), sums.prefix[kPxMost], (int64_t)sums.longs, (int32_t)gridDim.x, Q8);
        else
            return 0;
    }();
    const bool few = kFew && (int32_t)blockIdx.x >= split;
    const ChunkShares shares = [&]() -> ChunkShares {
        if constexpr (kFew) {
            const int64_t groups = sums.prefix[kPxMost];
            return few ? ck_shares(px_total(sums, pairs) - groups, (int32_t)gridDim.x - split) : ck_shares(groups, split);
        } else {
            return ck_shares(px_total(sums, pairs));
        }
    }();
    const int32_t cta = (int32_t)blockIdx.x - (few ? split : 0);
    const int64_t v0 = min(shares.total, cta * shares.share), v1 = min(shares.total, (cta + 1) * shares.share);
    Piece s;
    if constexpr (kShared)
        px_bind(p, sums, s, pairs, kFew ? kPxBeside : kPxAll, Q8);
    if constexpr (kFew) {
        const int64_t groups = sums.prefix[kPxMost];
        if (few) {
            // (costs from the groups' on)
            s.R = p.own_R;
            const bool have = ck_first<1>(p, sums, s, groups + v0, groups + v1);
            __syncthreads();
            if constexpr (Q8) {
                ShortMisc *sm = reinterpret_cast<ShortMisc *>(smem + p.few_misc);
                if (tid == 0)
                    short_init(sm);
                fence_proxy_async_smem();     // the loads overwrite the sums
                __syncthreads();
                short_body<D, 1, true>(p, ShortLayout{p.few_ring, p.few_raw, p.few_slots, p.few_o, p.few_ml, &p.few_k, &p.few_v}, sm,
                                          smem, s, have, groups + v1, cta, shares);
            } else {
                few_body<D>(p, smem, s, have, groups + v1, cta);
            }
            __syncthreads();
            if (warp == 1)
                tmem_dealloc(tmem, 512);
            return;
        }
        s.ne = s.ng;
    }
    const bool have0 = ck_first<NT>(p, sums, s, v0, v1);
    fence_proxy_async_smem();             // the loads overwrite the sums
    __syncthreads();
    auto is_long = [&](const Piece &x) { return !kMono && x.ntok > p.R; };

    if (warp == 0 || warp == 3) {
        // ============================================================ K / V loaders
        // Two warps, as issuing the copies of 16-token pages is what bounds a single one: the ring's
        // positions (K and V of a tile, in halves for d = 256) are theirs in turn.  A warp runs its loop together: lane u looks after positions 4 u .. 4 u + 3
        // of a tile, which lie in one page, and the lane of a page's first positions loads the page.
        // What lies past the block's last visible key, and pages whose id is outside the pool, is
        // loaded from a page past the pool: TMA fills zeros.  Exponent bytes come by ordinary loads two
        // tiles ahead (page ids three), as copies of their own would double the TMA's requests, and go
        // to shared memory as the multipliers that the converting warps need.
        const int me = warp == 0 ? 0 : 1;
        bool ok = true;
        const int32_t nring = Q8 ? nraw : nslot;
        uint32_t done = 0, fills = 0; // tiles loaded, ring slots filled by this warp
        uint32_t slot = me, phase = 0;
        const uint64_t pol_once = l2_policy_evict_first();
        const int32_t in_page = (1 << p.c.page_shift) - 1;
        const bool loads = ((lane * 4) & in_page) == 0;
        const bool needs_k = me == 0 || !Cfg::kByKind;    // (the first loader tells the softmax of both)
        for (bool have = have0; have && ok; have = ck_next<NT>(p, s, v1)) {
            const int32_t *bt = p.c.block_table + ck_table(p, s);
            auto needed = [&](int32_t t) { return t < s.t1 && ((t * kCkKeys + lane * 4) & ~in_page) < s.len; };
            auto page_of = [&](int32_t t) -> int32_t {
                return needed(t) ? __ldg(bt + ((t * kCkKeys + lane * 4) >> p.c.page_shift)) : -1;
            };
            auto checked = [&](int32_t id, int32_t t) -> int32_t {   // -1: none, or none in the pool
                if (id >= 0 && id < p.c.num_pages)
                    return id;
                if (needed(t))
                    set_status(p.status, SVP_DEV_BAD_CONTEXT);
                return -1;
            };
            auto exps_of = [&](int kv, int32_t t, int32_t id) -> uint32_t {   // of this lane's four rows
                if (!Q8 || id < 0)
                    return 0;
                const int64_t at = (((int64_t)id * p.c.hkv + s.g) << p.c.page_shift) + ((t * kCkKeys + lane * 4) & in_page);
                return __ldg(reinterpret_cast<const uint32_t *>((kv ? p.c.v_exp : p.c.k_exp) + at));
            };
            const bool once = s.nb == 1;      // no other block of the request reads these keys
            int32_t id = checked(page_of(s.t0), s.t0), id1 = checked(page_of(s.t0 + 1), s.t0 + 1), id2 = page_of(s.t0 + 2);
            uint32_t ek = needs_k ? exps_of(0, s.t0, id) : 0u, ek1 = needs_k ? exps_of(0, s.t0 + 1, id1) : 0u;
            uint32_t ev = exps_of(1, s.t0, id), ev1 = exps_of(1, s.t0 + 1, id1);
            for (int32_t t = s.t0; t < s.t1 && ok; ++t, ++done) {
                id2 = checked(id2, t + 2);
                const int32_t id3 = page_of(t + 3);
                const uint32_t ek2 = needs_k ? exps_of(0, t + 2, id2) : 0u, ev2 = exps_of(1, t + 2, id2);
                // the largest exponent of the tile's visible rows, at least 2^-60 (NaN rows apart)
                const int32_t left = s.len - t * kCkKeys - lane * 4;   // of this lane's rows, the visible
                auto top_of = [&](uint32_t e) -> uint32_t {
                    uint32_t top = 67;
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const uint32_t b = (e >> (8 * x)) & 0xffu;
                        top = max(top, x < left && b != 255u ? b : 0u);
                    }
                    return __reduce_max_sync(0xffffffffu, top);
                };
                uint32_t topk = 0, topv = 0;
                if constexpr (Q8) {
                    topv = top_of(ev);
                    if (needs_k) {
                        topk = top_of(ek);
                        if (me == 0 && lane == 0)
                            m->scales[done & 15] = make_float2(__uint_as_float(topk << 23), (float)((int32_t)topv - 127));
                    }
                }
                const int32_t page = id < 0 ? max(p.c.num_pages, 1) : id;
                for (int j = 0; j < NH; ++j) {
                    const int kv = Cfg::kByKind ? me : j, h = Cfg::kByKind ? 0 : me;
                    const CUtensorMap *tm = kv ? &p.tm_v : &p.tm_k;
                    const uint32_t full = Q8 ? bar_rfull(slot) : bar_full(slot);
                    int got = 1;
                    if (lane == 0)
                        got = mbar_wait(Q8 ? bar_rempty(slot) : bar_empty(slot), phase ^ 1u, abort_flag);
                    if (!(ok = __shfl_sync(0xffffffffu, got, 0) != 0))
                        break;
                    if constexpr (Q8) {
                        const uint32_t dst = sbase + p.off_raw + slot * Cfg::kRawSlot;
                        if (loads) {
                            if (once)
                                tma_load_4d_hint(dst + lane * 4 * DH, tm, full, h * DH, 0, s.g, page, pol_once);
                            else
                                tma_load_4d(dst + lane * 4 * DH, tm, full, h * DH, 0, s.g, page);
                        }
                        // 2^(b - top) in fp16 (NaN for byte 255, 0 past the last visible key)
                        uint32_t mul[4];
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const uint32_t b = ((kv ? ev : ek) >> (8 * x)) & 0xffu;
                            const int32_t down = (int32_t)(kv ? topv : topk) - (int32_t)b;
                            const uint32_t f = b == 255u ? 0x7e00u
                                               : down <= 14 ? (uint32_t)(15 - down) << 10
                                               : down <= 24 ? 1u << (24 - down) : 0u;
                            mul[x] = x < left ? f : 0u;
                        }
                        ck_st_v2(dst + Cfg::kRaw + lane * 8, mul[0] | (mul[1] << 16), mul[2] | (mul[3] << 16));
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive_expect_tx(full, (uint32_t)Cfg::kRaw);
                    } else {
                        const uint32_t dst = sbase + p.off_ring + slot * Cfg::kSlot;
                        if (lane == 0)
                            mbar_arrive_expect_tx(full, (uint32_t)Cfg::kSlot);
                        __syncwarp();
                        if (loads) {
#pragma unroll
                            for (int c = 0; c < DH / 64; ++c) {
                                const uint32_t at = dst + c * kCkSub + lane * 512;
                                if (once)
                                    tma_load_4d_hint(at, tm, full, h * DH + c * 64, 0, s.g, page, pol_once);
                                else
                                    tma_load_4d(at, tm, full, h * DH + c * 64, 0, s.g, page);
                            }
                        }
                    }
                    __syncwarp();
                    ++fills;
                    if ((slot += 2) >= (uint32_t)nring) {
                        slot -= nring;
                        phase ^= 1u;
                    }
                }
                ek = ek1;
                ek1 = ek2;
                ev = ev1;
                ev1 = ev2;
                id = id1;
                id1 = id2;
                id2 = id3;
            }
        }
        // every load lands (and, of the bf16 ring, every release by the tensor core) before the
        // CTA's shared memory is given back; a fill that did not happen is not waited for
        if (lane == 0) {
            volatile int drain = 0;
            // Of this warp's positions 2 x + me, those that no later one has waited for: of its own, nring
            // further on, or of the other warp's last.
            const int32_t seen = 2 * ((int32_t)fills - 1) + (me == 0 && ok ? 1 : 0) - nring;
            for (uint32_t x = seen < 0 ? 0u : (uint32_t)seen / 2 + 1; x < fills; ++x) {
                const uint32_t sl = (2 * x + me) % nring, ph = ((2 * x + me) / nring) & 1u;
                mbar_wait(Q8 ? bar_rfull(sl) : bar_full(sl), ph, &drain);
                if (!Q8 && ok)
                    mbar_wait(bar_empty(sl), ph, abort_flag);
            }
        }
        __syncwarp();
    } else if (warp == 1 || warp == 2) {
        // ============================================================ MMA issuers
        // A thread's waits queue behind the MMAs it has issued, so one issuer alone leaves the tensor
        // pipe idle between them: two warps issue.  d <= 128: warp 1 + a issues S_a and PV_a (its own
        // next wait, for the P that follows that S, could not end earlier anyway), and in short pieces
        // only looks after every other tile.  d = 256: warp 1 issues S, warp 2 PV.  Both warps see every
        // ring slot filled and both release it (a parity wait may not skip a phase).  The warps run
        // their loops together (they clear V rows together); lane 0 issues.
        const int me = warp - 1;
        // bf16 operands, or fp16 ones (type bits 0) made from 8-bit pages
        const uint32_t types = Q8 ? ~((1u << 7) | (1u << 10)) : ~0u;
        const uint32_t idesc_s = idesc_bf16_f32(128, 128, false, false) & types;
        const uint32_t idesc_o = idesc_bf16_f32(128, DH, false, true) & types;
        uint32_t nq = 0, q_loads = 0;         // query tiles used and loaded
        uint32_t npiece = 0, nturn = 0;
        uint32_t nsp[2] = {0, 0}, no = 0;     // uses of S / P buffer a, and of this warp's O, so far
        bool ok = true;
        uint32_t slot = 0, phase = 0;         // ring position
        auto step = [&]() {
            if (++slot == (uint32_t)nslot) {
                slot = 0;
                phase ^= 1u;
            }
        };
        auto wait_all = [&](uint32_t bar, uint32_t parity) {
            return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag));
        };
        // Long pieces: the two issuers take turns, PV of a tile and S of the next at a time, warp 1 first.
        // Left to share the pipe they keep in step: both tiles' MMAs at once, then both softmaxes.
        auto turn = [&]() -> bool {
            const uint32_t n = nturn++;
            return me == 0 ? n == 0 || wait_all(bar_turn(0), (n - 1) & 1u) : wait_all(bar_turn(1), n & 1u);
        };
        // NH slots of the other warp's: seen and released
        auto pass = [&]() -> bool {
            for (int h = 0; h < NH; ++h) {
                if (!wait_all(bar_full(slot), phase))
                    return false;
                if (lane == 0)
                    mbar_arrive(bar_empty(slot));
                step();
            }
            return true;
        };
        auto my_jobs = [&](const Piece &x) -> int32_t {   // tiles of the piece that this warp works on
            const int32_t nt = x.t1 - x.t0;
            return kMono || is_long(x) ? nt : (nt + 1 - me) >> 1;
        };
        auto load_q = [&](const Piece &x) {
            if (kMono ? me != 0 : my_jobs(x) == 0)
                return;
            if (lane == 0) {
                mbar_arrive_expect_tx(bar_q(me), (uint32_t)((D / 64) * 128 * p.G * p.Rb));
                for (int c = 0; c < D / 64; ++c)
                    tma_load_3d(sbase + (me * (D / 64) + c) * p.qsub, &p.tm_q, bar_q(me), c * 64, x.g * p.G,
                                x.off + x.tb0 + (is_long(x) ? me * p.R : 0));
            }
            __syncwarp();
            ++q_loads;
        };
        // S of the tile at the ring position; give: the turn passes on before its last products, as the
        // arrival queues behind the ones before it and the other issuer takes a while to wake
        auto issue_s = [&](int buf, bool give) -> bool {
            for (int h = 0; h < NH; ++h) {
                if (!wait_all(bar_full(slot), phase))
                    return false;
                tc_fence_after();
                if (ck_elect()) {
                    const uint64_t qd = sw128_desc(sbase + (me * (D / 64) + h * 2) * p.qsub, 16, 1024);
                    const uint64_t kd = sw128_desc(sbase + p.off_ring + slot * Cfg::kSlot, 16, 1024);
                    const uint32_t qs16 = (uint32_t)p.qsub >> 4;
#pragma unroll
                    for (int ks = 0; ks < DH / 16; ++ks) {
                        if (ks == kGiveAt && give)
                            mbar_arrive(bar_turn(me ^ 1));
                        tc_mma_ss(tmem + buf * 128, qd + (uint64_t)((ks >> 2) * qs16 + (ks & 3) * 2),
                                  kd + (uint64_t)((ks >> 2) * (kCkSub >> 4) + (ks & 3) * 2), idesc_s,
                                  (h | ks) ? 1u : 0u);
                    }
                    if (h == NH - 1)
                        tc_commit(bar_s(buf));
                    tc_commit(bar_empty(slot));
                }
                step();
            }
            __syncwarp();
            return true;
        };
        bool have_next = false;
        auto issue_pv = [&](int buf, int ob, int32_t kvalid, bool first, bool last, bool lng) -> bool {
            uint32_t sl[NH];
            for (int h = 0; h < NH; ++h) {
                if (!wait_all(bar_full(slot), phase))
                    return false;
                sl[h] = slot;
                step();
            }
            // rows of the last page past the last visible key may hold anything, and P = 0 does not hide
            // a NaN: they are cleared (whole pages past it are zeros already, and the converting warps'
            // multipliers clear theirs)
            const int32_t rest = kvalid & ((1 << p.c.page_shift) - 1);
            if (!Q8 && kvalid < kCkKeys && rest) {
                const int32_t rows = (1 << p.c.page_shift) - rest;
                for (int h = 0; h < NH; ++h)
                    for (int32_t x = lane; x < rows * (DH / 8); x += 32) {
                        const int32_t r = kvalid + x / (DH / 8), c = x % (DH / 8);
                        st_shared_v4(sbase + p.off_ring + sl[h] * Cfg::kSlot + (c >> 3) * kCkSub + r * 128 +
                                         (c & 7) * 16, 0u, 0u, 0u, 0u);
                    }
                fence_proxy_async_smem();
                __syncwarp();
            }
            if (first && no > 0 && !wait_all(bar_ofree(ob), (no - 1) & 1u))
                return false;
            if (!wait_all(bar_p(buf), nsp[buf] & 1u))
                return false;
            ++nsp[buf];
            if (!kMono && last) {
                // this warp's last P of the piece: all its S are done and its query tile may be replaced
                have_next = ck_next<NT>(p, s, v1);
                if (have_next)
                    load_q(s);
            }
            if (lng && !turn())
                return false;
            tc_fence_after();
            if (ck_elect()) {
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    const uint64_t vd = sw128_desc(sbase + p.off_ring + sl[h] * Cfg::kSlot, kCkSub, 1024);
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks)   // 16 keys = 8 TMEM columns of P a step
                        ck_mma_ts(tmem + 256 + ob * D + h * DH, tmem + buf * 128 + ks * 8, vd + (uint64_t)(ks * 128),
                                  idesc_o, (!first || ks) ? 1u : 0u);
                    tc_commit(bar_empty(sl[h]));
                }
                if (kMono)
                    tc_commit(bar_pv(buf));
                if (last)
                    tc_commit(bar_o(ob));
            }
            __syncwarp();
            return true;
        };
        bool have = have0;
        if (have)
            load_q(s);
        while (have && ok) {
            const int32_t nt = s.t1 - s.t0, mine = my_jobs(s);
            const bool lng = is_long(s);
            if (mine > 0 && (!kMono || me == 0)) {
                // (8-bit pages: until the softmax warps have made it fp16)
                if (!(ok = wait_all(Q8 ? bar_qc(me) : bar_q(me), nq & 1u)))
                    break;
                ++nq;
            }
            // (from the last P on, s is the next piece: what the loop needs of this one is kept here)
            int32_t kvalid = s.len - s.t0 * kCkKeys;      // keys of tile t that the block sees
            for (int32_t t = 0; t < nt; ++t, kvalid -= kCkKeys) {
                if (kMono) {
                    const int buf = t & 1;
                    if (me == 0) {
                        // the buffer's last P has been read
                        if (!(ok = nsp[buf] == 0 || wait_all(bar_pv(buf), (nsp[buf] - 1) & 1u)) ||
                            !(ok = issue_s(buf, false)))
                            break;
                        ++nsp[buf];
                        if (t == nt - 1 && lane == 0)
                            tc_commit(bar_sdone);
                        if (!(ok = pass()))
                            break;
                    } else if (!(ok = pass()) || !(ok = issue_pv(buf, 0, kvalid, t == 0, t == nt - 1, false))) {
                        break;
                    }
                } else if (lng) {
                    // (the K wait is inside the turn: the other issuer needs the same tile)
                    if ((t == 0 && !(ok = turn())) || !(ok = issue_s(me, true)) ||
                        !(ok = issue_pv(me, me, kvalid, t == 0, t == nt - 1, true)))
                        break;
                    if (t == nt - 1 && lane == 0)
                        mbar_arrive(bar_turn(me ^ 1));
                } else if ((t & 1) == me) {
                    if (!(ok = issue_s(me, false)) || !(ok = issue_pv(me, me, kvalid, t < 2, t + 2 >= nt, false)))
                        break;
                } else if (!(ok = pass()) || !(ok = pass())) {
                    break;
                }
            }
            if (!ok)
                break;
            if (mine > 0)
                ++no;
            if (kMono || mine == 0) {
                have_next = ck_next<NT>(p, s, v1);
                if (kMono && me == 0 && !(ok = wait_all(bar_sdone, npiece & 1u)))
                    break;
                if (have_next)
                    load_q(s);
            }
            ++npiece;
            have = have_next;
        }
        if (lane == 0) {
            volatile int drain = 0;
            tc_commit(bar_drain(me));
            mbar_wait(bar_drain(me), 0, &drain);
            for (uint32_t k = nq; k < q_loads; ++k)   // a query tile on its way when a wait gave up
                mbar_wait(bar_q(me), k & 1u, &drain);
        }
        __syncwarp();
    } else if (warp >= Cfg::kSoftWarp0 && warp < Cfg::kConvWarp0) {
        // ============================================================ softmax, one row a thread
        const int a = (warp - Cfg::kSoftWarp0) >> 2;
        const int r = (warp & 3) * 32 + lane;             // row of the tile = TMEM lane
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t to0 = tmem + lane_off + 256;
        uint32_t ntile = 0, nq = 0;                       // KV tiles and query tiles of earlier pieces
        uint32_t ns_[2] = {0, 0}, no_[2] = {0, 0}, nml = 0;
        bool ok = true, owe = false;
        auto wait_all = [&](uint32_t bar, uint32_t parity) {
            return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag));
        };
        for (bool have = have0; have; have = ck_next<NT>(p, s, v1)) {
            const bool lng = is_long(s);
            const int32_t nt = s.t1 - s.t0;
            const int32_t tok = (lng ? a * p.R : 0) + r / p.G;      // token of the block
            const bool live = r < p.G * p.R && tok < s.ntok;
            const bool warp_live = __any_sync(0xffffffffu, live);
            const int32_t last = live ? ck_last(s, tok) : -1;        // last visible key
            const int32_t all = ck_last(s, lng ? a * p.R : 0);       // last key that every row sees
            const uint32_t to = to0 + (kMono ? 0 : a * D);
            float m_ref = -INFINITY, l = 0.0f;
            int32_t done = 0;                                        // tiles of this warpgroup so far
            float cl2 = p.scale_log2;
            float e_first = 0.0f;                                    // 8-bit pages: E of V in its first tile
            if (Q8 && (lng || kMono || a < nt)) {
                // This row of the query in fp16, times the power of two that takes its largest magnitude
                // to 2^14 or more
                if (!(ok = wait_all(bar_q(a), nq & 1u)))
                    break;
                ++nq;
                if (live) {
                    const uint32_t line = sbase + a * (D / 64) * p.qsub + r * 128;
                    uint32_t top = 0;
                    // (32 columns at a time: all reads, then what is done with them)
#pragma unroll 1
                    for (int pass = 0; pass < 2; ++pass) {
                        const int32_t shift = ck_q_shift(top);
                        const float f = ck_pow2(shift);
#pragma unroll 1
                        for (int x = 0; x < D / 8; x += 4) {
                            int4 w[4];
#pragma unroll
                            for (int y = 0; y < 4; ++y)
                                w[y] = ld_shared_i4(line + (x >> 3) * p.qsub + ((((x & 7) + y) ^ (r & 7)) << 4));
#pragma unroll
                            for (int y = 0; y < 4; ++y) {
                                const uint32_t v[4] = {(uint32_t)w[y].x, (uint32_t)w[y].y, (uint32_t)w[y].z, (uint32_t)w[y].w};
                                if (pass == 0) {
#pragma unroll
                                    for (int z = 0; z < 4; ++z)
                                        top = max(top, max(v[z] & 0x7fffu, (v[z] >> 16) & 0x7fffu));
                                } else {
                                    uint32_t u[4];
#pragma unroll
                                    for (int z = 0; z < 4; ++z)
                                        u[z] = ck_pack_f16x2(bf16_lo(v[z]) * f, bf16_hi(v[z]) * f);
                                    st_shared_v4(line + (x >> 3) * p.qsub + ((((x & 7) + y) ^ (r & 7)) << 4), u[0], u[1], u[2], u[3]);
                                }
                            }
                        }
                        if (pass == 1)
                            cl2 *= ck_pow2(-shift);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar_qc(a));
            }
            for (int32_t t = (lng || kMono) ? 0 : a; t < nt; t += (lng || kMono) ? 1 : 2, ++done) {
                const int buf = kMono ? (t & 1) : a;
                const uint32_t ts = tmem + lane_off + buf * 128;
                if (!(ok = wait_all(bar_s(buf), ns_[buf] & 1u)))
                    break;
                ++ns_[buf];
                // Barriers are waited for by parity, so no phase may be skipped, nor waited for when the
                // next may have completed.  O_1 of an earlier short piece, which the first warpgroup
                // read: no later phase can complete before the arrival below.
                if (owe && !(ok = wait_all(bar_o(1), (no_[1] - 1) & 1u)))
                    break;
                owe = false;
                // d = 256: PV of the tile before, into the same O, is waited for before a rescale and before
                // the arrival below (which PV of this tile needs; the pipe has S of the next to go on with)
                bool pv_seen = !kMono || t == 0;
                tc_fence_after();
                if (warp_live) {
                    const int32_t k0 = (s.t0 + t) * kCkKeys;
                    const bool masked = k0 + kCkKeys - 1 > all;
                    const int32_t kmax = last - k0;
                    // 8-bit pages: K and V of the tile are in units of 2^E; the probabilities take over V's
                    // (P 2^E V, against a reference of s c + E, so the accumulator needs no other), and
                    // the sum gives it back, relative to the first tile's
                    float ct = cl2, ev = 0.0f;
                    if constexpr (Q8) {
                        const float2 sc = m->scales[(ntile + t) & 15];
                        ct = fmaxf(ct * sc.x, FLT_MIN);   // (0 times the -inf of a hidden key would be NaN)
                        ev = sc.y;
                        if (done == 0)
                            e_first = ev;
                    }
                    // Without a mask, and with a reference that still holds, the scores are read once: where the
                    // registers hold a row's P (4096 rows on 8192 keys 507 us, read twice 570)
                    constexpr bool kOnce = !Q8;
                    float sum = 0.0f;
                    if (!kOnce || masked || done == 0 || !ck_row_once<Q8>(ts, ct, m_ref - ev, 32768.0f, live, sum)) {
                        const float tmax = (masked ? ck_row_max<true>(ts, kmax) : ck_row_max<false>(ts, kmax)) * ct + ev;
                        // the reference moves when a score lies more than 2^8 above it (or there is none yet); it is
                        // the largest score less kLift
                        constexpr float kLift = Q8 ? kCkLift : 0.0f;
                        if (__any_sync(0xffffffffu,
                                       live && (tmax > m_ref + (kCkSlack + kLift) || (m_ref == -INFINITY && tmax != m_ref)))) {
                            const float m_new = fmaxf(m_ref, tmax - kLift);
                            if (done > 0) {
                                const float alpha = m_ref == -INFINITY ? 0.0f : fast_exp2(m_ref - m_new);
                                if (!pv_seen && !(ok = wait_all(bar_pv(buf ^ 1), (ns_[buf ^ 1] - 1) & 1u)))
                                    break;
                                pv_seen = true;
                                tc_fence_after();
#pragma unroll 1
                                for (int cc = 0; cc < D / 32; ++cc) {
                                    uint32_t ov[32];
                                    tmem_ld32(to + cc * 32, ov);
                                    tmem_wait_ld();
#pragma unroll
                                    for (int e = 0; e < 32; ++e)
                                        ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
                                    tmem_st32(to + cc * 32, ov);
                                }
                                l *= alpha;
                            }
                            m_ref = m_new;
                        }
                        const float mm = (m_ref == -INFINITY ? 0.0f : m_ref) - ev;
                        sum = masked ? ck_row_exp<true, Q8>(ts, kmax, ct, mm) : ck_row_exp<false, Q8>(ts, kmax, ct, mm);
                    }
                    l += Q8 ? sum * ck_pow2((int32_t)(e_first - ev)) : sum;
                    tmem_wait_st();
                }
                if (!pv_seen && !(ok = wait_all(bar_pv(buf ^ 1), (ns_[buf ^ 1] - 1) & 1u)))
                    break;
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar_p(buf));
            }
            if (!ok)
                break;
            const bool both = !kMono && !lng && nt > 1;   // two accumulators of one query tile
            float o_scale = 1.0f;                         // O and m in units of 1 from here on
            if constexpr (Q8) {
                o_scale = ck_pow2((int32_t)(e_first - kCkLift));
                l *= ck_pow2(-(int32_t)kCkLift);
                m_ref += kCkLift - e_first;
                ntile += (uint32_t)nt;
            }
            if (both && a == 1) {
                // (m, l) to the first warpgroup, which joins the two halves
                if (nml > 0 && !(ok = wait_all(bar_mlfree, (nml - 1) & 1u)))
                    break;
                m->ml[r] = make_float2(m_ref, l);
                if (Q8 && r == 0)
                    m->o_scale = o_scale;          // (of all its live rows; row 0 is one)
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar_ml);
                owe = true;
            }
            if (a == 0 || lng) {
                if (!(ok = wait_all(bar_o(a), no_[a] & 1u)) || (both && !(ok = wait_all(bar_o(1), no_[1] & 1u))))
                    break;
                tc_fence_after();
                float f0 = 1.0f, f1 = 0.0f;
                if (both) {
                    if (!(ok = wait_all(bar_ml, nml & 1u)))
                        break;
                    const float2 o = m->ml[r];
                    const float o1_scale = Q8 ? m->o_scale : 1.0f;
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(bar_mlfree);
                    // a half without a visible key has l = 0 and is left out whatever its O holds (not so one whose
                    // weight underflows: its O may be NaN)
                    if (o.y != 0.0f) {
                        const float mx = fmaxf(m_ref, o.x);
                        f0 = m_ref == -INFINITY ? 0.0f : fast_exp2(m_ref - mx);
                        f1 = fast_exp2(o.x - mx);
                        l = l * f0 + o.y * f1;
                        m_ref = mx;
                        f1 = fmaxf(f1 * o1_scale, FLT_MIN);
                    }
                }
                f0 *= o_scale;
                const bool whole = s.t0 == 0 && s.t1 == s.nt && !ck_kept(s);   // its result is the output's
                const int32_t row = s.off + s.tb0 + tok, head = s.g * p.G + r % p.G;
                const int32_t slot = 2 * cta + (s.t0 > 0 ? 0 : 1);
                int64_t prow = (int64_t)slot * Cfg::kPartRows + (lng ? a * 128 : 0) + r;
                float *part_o = p.part_o;
                float2 *part_ml = p.part_ml;
                if constexpr (kShared) {
                    if (s.t0 == 0 && s.t1 == s.nt) {
                        prow = px_place(p, s.group, row, head);
                        part_o = p.place_o;
                        part_ml = p.place_ml;
                    }
                }
                const float inv = 1.0f / l;
                if (warp_live) {
#pragma unroll 1
                    for (int cc = 0; cc < D / 32; ++cc) {
                        uint32_t ov[32];
                        tmem_ld32(to + cc * 32, ov);
                        if (both) {
                            uint32_t ow[32];
                            tmem_ld32(to + D + cc * 32, ow);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                ov[e] = __float_as_uint(__uint_as_float(ov[e]) * f0 +
                                                        (f1 != 0.0f ? __uint_as_float(ow[e]) * f1 : 0.0f));
                        } else {
                            tmem_wait_ld();
                            if (Q8) {
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    ov[e] = __float_as_uint(__uint_as_float(ov[e]) * f0);
                            }
                        }
                        if (!live)
                            continue;
                        if (whole) {
                            uint32_t pk[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                pk[e] = pack_bf16x2(__uint_as_float(ov[2 * e]) * inv, __uint_as_float(ov[2 * e + 1]) * inv);
                            uint16_t *dst = reinterpret_cast<uint16_t *>(p.out) + ((int64_t)row * p.hq + head) * D + cc * 32;
                            if (p.out32) {
                                ck_store8(dst, pk);
                                ck_store8(dst + 16, pk + 8);
                            } else {
#pragma unroll
                                for (int v = 0; v < 4; ++v)
                                    reinterpret_cast<uint4 *>(dst)[v] =
                                        make_uint4(pk[4 * v], pk[4 * v + 1], pk[4 * v + 2], pk[4 * v + 3]);
                            }
                        } else {
                            float *dst = part_o + prow * D + cc * 32;
#pragma unroll
                            for (int v = 0; v < 4; ++v)
                                ck_store8(dst + 8 * v, ov + 8 * v);
                        }
                    }
                    if (live) {
                        if (!whole)
                            part_ml[prow] = make_float2(m_ref, l);
                        else if (p.lse)
                            p.lse[(int64_t)row * p.hq + head] = (m_ref + __log2f(l)) * 0.69314718055994531f;
                    }
                }
                if (!kShared && !whole && s.t0 == 0 && a == 0 && r == 0) {
                    // this CTA has the pair's first piece: CTAs up to the owner of its last tile have the rest
                    ChunkDesc d;
                    d.np = ck_owner(shares, s.base + (int64_t)s.wt * (kStartKeys + (int64_t)kCkKeys * (s.nt - 1))) - cta + 1;
                    d.row0 = s.off + s.tb0;
                    d.ntok = s.ntok;
                    d.g = s.g;
                    p.desc[cta] = d;
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar_ofree(a));
                    if (both)
                        mbar_arrive(bar_ofree(1));
                }
            }
            // uses of the accumulators, as the issuer counts them
            ++no_[0];
            if (!kMono && (lng || nt > 1))
                ++no_[1];
            if (both)
                ++nml;
        }
    } else if (Q8 && warp >= Cfg::kConvWarp0) {
        // ============================================================ codes -> fp16 tiles
        // A thread takes 16 codes of one row at a time, its neighbours the rest of the row.
        if constexpr (Q8) {
            constexpr int CPR = DH / 16;                  // 16-code chunks a row
            constexpr int RPI = 32 * Cfg::kConvWarps / CPR, IT = 128 / RPI;   // rows a turn, turns
            const int ct = tid - Cfg::kConvWarp0 * 32;
            const int c = ct % CPR, row0 = ct / CPR;
            // which half of its 16 codes a thread takes first: the lanes of one access then cover all banks,
            // in the raw rows as in the swizzled ones
            const int odd = (DH == 128 ? (c >> 2) ^ row0 : row0 >> 1) & 1;
            const uint32_t src = row0 * DH + c * 16 + odd * 8, src2 = row0 * DH + c * 16 + (odd ^ 1) * 8;
            const uint32_t line = (c >> 2) * kCkSub + row0 * 128;
            const uint32_t out = line + (((2 * (c & 3) + odd) ^ (row0 & 7)) << 4);
            const uint32_t out2 = line + (((2 * (c & 3) + (odd ^ 1)) ^ (row0 & 7)) << 4);
            uint32_t pos = 0, halves = 0;                 // ring positions done, of all pieces
            for (bool have = have0; have; have = ck_next<NT>(p, s, v1))
                halves += (uint32_t)(s.t1 - s.t0) * 2 * NH;
            uint32_t slot = 0, phase = 0, rslot = 0, rphase = 0;
            bool ok = true;
            for (; pos < halves; ++pos) {
                const bool got = mbar_wait(bar_rfull(rslot), rphase, abort_flag) &&
                                 mbar_wait(bar_empty(slot), phase ^ 1u, abort_flag);
                if (!(ok = __all_sync(0xffffffffu, got)))
                    break;
                const uint8_t *raw = smem + p.off_raw + rslot * Cfg::kRawSlot;
                const uint32_t dst = sbase + p.off_ring + slot * Cfg::kSlot;
                // all reads first: each takes long beside the tensor core's, and none may pass a write
                uint2 w[IT], w2[IT];
                uint32_t mul[IT];
#pragma unroll
                for (int it = 0; it < IT; ++it) {
                    w[it] = *reinterpret_cast<const uint2 *>(raw + src + it * (RPI * DH));
                    w2[it] = *reinterpret_cast<const uint2 *>(raw + src2 + it * (RPI * DH));
                    mul[it] = *reinterpret_cast<const uint16_t *>(raw + Cfg::kRaw + (it * RPI + row0) * 2) * 0x10001u;
                }
#pragma unroll
                for (int it = 0; it < IT; ++it) {
                    if (mul[it] == 0u)                // (the codes may be NaN, which 0 would not hide)
                        w[it] = w2[it] = make_uint2(0u, 0u);
                    uint32_t x[8];
                    ck_codes(w[it].x, mul[it], x[0], x[1]);
                    ck_codes(w[it].y, mul[it], x[2], x[3]);
                    ck_codes(w2[it].x, mul[it], x[4], x[5]);
                    ck_codes(w2[it].y, mul[it], x[6], x[7]);
                    st_shared_v4(dst + out + it * (RPI * 128), x[0], x[1], x[2], x[3]);
                    st_shared_v4(dst + out2 + it * (RPI * 128), x[4], x[5], x[6], x[7]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar_rempty(rslot));
                    mbar_arrive(bar_full(slot));
                }
                if (++slot == (uint32_t)nslot) {
                    slot = 0;
                    phase ^= 1u;
                }
                if (++rslot == (uint32_t)nraw) {
                    rslot = 0;
                    rphase ^= 1u;
                }
            }
            // the tensor core's releases land before the CTA's shared memory is given back
            if (lane == 0 && ok) {
                const uint32_t first = pos > (uint32_t)nslot ? pos - nslot : 0u;
                for (uint32_t k = first; k < pos; ++k)
                    mbar_wait(bar_empty((int)(k % nslot)), (k / nslot) & 1u, abort_flag);
            }
            __syncwarp();
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (*abort_flag && tid == 0)
        set_status(p.status, SVP_DEV_TIMEOUT);
    if (warp == 1)
        tmem_dealloc(tmem, 512);
}

}  // namespace svp
