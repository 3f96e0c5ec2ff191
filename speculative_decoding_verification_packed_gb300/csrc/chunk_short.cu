// chunk_short.cu -- decode tokens and short candidate blocks over 8-bit pages.
//
// The same operator as chunk_tc.cu, for calls whose requests have at most 16 query rows a KV head
// (G heads times w tokens) and d <= 128, where the pages' bytes bound the time.  There tcgen05 does
// not pay: its operands come from shared memory in 16 bits, so every code is read, widened, written
// and read again by the tensor core, more shared-memory traffic than the bytes' time allows (64
// requests x 18000 tokens, 8 KV heads, d 128: 640 us).  Here codes go from shared memory to registers,
// are widened there (cvt: two codes an instruction), and warp-level m16n8k16 products take them as
// they are: 363 us, 6.6 TB/s with 16-token pages and 344 us with 128-token ones.
//
// Keys are the products' 16-row side and query rows the 8-column side,
//   S^T (16 keys x 8 rows) = K Q^T,   O^T (16 of d x 8 rows) += V^T P^T,
// as the rate of these products bounds the kernel next (with rows on the 16-row side, half of them
// empty for G = 4 tokens, the same call took 467 us when this way took 381).  Eight warps share the
// 128 positions of a KV tile, 16 each.  A warp keeps Q (fp16, the row's power of two taken out), its rows'
// running maximum and sum and its O in registers; the warps join at the end of a piece through shared
// memory.  NB = 1 or 2 blocks of 8 rows (488 us with 16 rows, bound by the products).  d = 64 takes 330 us
// for half the bytes: the chain of a tile is as long, and copies of 1 KB come no faster than those
// of 2 KB (262 us with 128-token pages).  d is taken in the order in which a thread finds it: for S,
// thread q of a quad has d = D/4 q .. of its key in one read; for O, d = D/8 n + i belongs to row n of
// the product's half i.  P^T turns from accumulator to operand by movmatrix.
// An 8-bit row's power of two multiplies its row of S^T; V's goes into the exponent,
//   P' = 2^(s c + e_key - m),  O += P' codes,  l += P' 2^(e_ref - e_key),
// with m the running maximum of s c + e_key (less kCkLift), so that P' stays within fp16 whatever the
// exponents (it is rounded to fp16 because the products take 16 bits; scores, m, l and O are fp32).
// e_ref, one a warp, keeps l in range: 0 until a visible row that is not all zeros has e_key < -kShSpan,
// then kShSpan above the smallest e_key so far.  With P' < 2^15 a term is below 2^79, and 2^20
// keys add up to less than 2^100; P' = 2^7 of a key whose e_key is 2^100 above the smallest, or 2^100 above 1
// where none is below it, counts 2^-93 or more, far from the end of fp32's range.  The test shares
// the vote on m; one of its own cost 3 us more, and the factors made by the V loader 32.
// (Without e_ref, when rows of zeros made l infinite, it took 358, and 16 rows 469.)  Where most tiles have
// rows of zeros, which are looked at again in each, it takes 480, and 16 rows 682.
// Pieces, their split over the CTAs and the joining of split pairs are those of chunk_tc.cu.
#include <algorithm>
#include <cstring>

#include "chunk_pieces.cuh"

namespace svp {

constexpr int kShWarps = 8;           // computing warps; then a K and a V loader
constexpr int kShThreads = 32 * (kShWarps + 2);
constexpr int kShSlots = 16;          // ring slots at most
constexpr float kShSpan = 64.0f;      // e_ref - e_key, at most
constexpr float kShNan = -128.0f, kShZero = -127.0f;   // e_key of a value row that stands for NaN, for zeros
// e_key that rows of zeros get: above -kShSpan, so that they do not move e_ref, and low, so that one that takes
// most of the weight leaves fp16's range to the others (at 0, one of 2^24 times their weight took their digits)
constexpr float kShZeros = -60.0f;

struct ShortMisc {
    uint64_t bars[2 * kShSlots];
    int32_t abort_flag, pad;
    int64_t warp_tot[12];
    int32_t nan_at[kShWarps];         // position of the first value row of a warp's that stands for NaN
    float2 ml[kShWarps][16];          // [warp][row of its group]
};

template <int D, int NB>
struct ShortCfg {
    static constexpr int kRaw = kCkKeys * D;
    static constexpr int NI = D / 8;                        // d of one row of an O product's halves
    static constexpr int KS = D / 16;                       // k steps of S
    static constexpr int kRed = kShWarps * 8 * NB * (D + 8) * 4;   // the warps' O, rows padded
};

// C += A B, fp16 operands, fp32 accumulators (m16n8k16).
__device__ __forceinline__ void sh_mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A transposed 8 x 8 block of fp16 pairs.
__device__ __forceinline__ uint32_t sh_turn(uint32_t x)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// Four codes to two fp16 pairs.
__device__ __forceinline__ void sh_codes(uint32_t w, uint32_t &lo, uint32_t &hi)
{
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

// 16-byte chunk c of row `row` in a raw tile (128-byte rows with 128-byte swizzle, 64 with 64).
template <int D>
__device__ __forceinline__ uint32_t sh_chunk(int row, int c)
{
    return D == 128 ? row * 128 + ((c ^ (row & 7)) << 4) : row * 64 + ((c ^ ((row >> 1) & 3)) << 4);
}

template <int D, int NB>
__global__ void __launch_bounds__(kShThreads, 1) chunk_short_kernel(const __grid_constant__ ChunkParams p)
{
    using Cfg = ShortCfg<D, NB>;
    constexpr int NI = Cfg::NI, KS = Cfg::KS;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    ShortMisc *m = reinterpret_cast<ShortMisc *>(smem + p.off_misc);
    const uint32_t bar0 = smem_u32(m->bars);
    auto bar_full = [&](uint32_t s) { return bar0 + 8u * s; };
    auto bar_empty = [&](uint32_t s) { return bar0 + 8u * (kShSlots + s); };
    volatile int *abort_flag = &m->abort_flag;
    const uint32_t nslot = (uint32_t)p.nslot;
    if (tid == 0) {
        for (int s = 0; s < kShSlots; ++s) {
            mbar_init(bar_full(s), 1);
            mbar_init(bar_empty(s), kShWarps);
        }
        mbar_fence_init();
        m->abort_flag = 0;
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

    if (warp >= kShWarps) {
        // ============================================================ K loader, V loader
        // Even ring slots hold K, odd ones V.  Lane u looks after positions 4 u .. 4 u + 3 of a tile; the
        // lane of a page's first positions loads the page; pages that are not needed or not in the
        // pool are loaded from past the pool (zeros).  The rows' exponents go beside the codes as fp32:
        // K's as factors, V's as exponents (kShNan for byte 255).
        const int kv = warp - kShWarps;
        const CUtensorMap *tm = kv ? &p.tm_v : &p.tm_k;
        const uint8_t *exps = kv ? p.c.v_exp : p.c.k_exp;
        const uint64_t pol = l2_policy_evict_first();       // each byte is read once
        const int32_t in_page = (1 << p.c.page_shift) - 1;
        const bool loads = ((lane * 4) & in_page) == 0;
        uint32_t slot = kv, phase = 0, done = 0;
        bool ok = true;
        for (bool have = have0; have && ok; have = ck_next<1>(p, s, v1)) {
            const int32_t *bt = p.c.block_table + (int64_t)s.i * p.c.max_pages;
            constexpr int32_t kNone = INT32_MIN;   // (a table may hold it too: see checked)
            auto page_of = [&](int32_t t) -> int32_t {
                const int32_t at = t * kCkKeys + lane * 4;
                return t >= s.t1 || (at & ~in_page) >= s.len ? kNone : __ldg(bt + (at >> p.c.page_shift));
            };
            auto needed = [&](int32_t t) { return t < s.t1 && ((t * kCkKeys + lane * 4) & ~in_page) < s.len; };
            auto checked = [&](int32_t id, int32_t t) -> int32_t {
                if (id >= 0 && id < p.c.num_pages)
                    return id;
                if (id != kNone || needed(t))
                    set_status(p.status, SVP_DEV_BAD_CONTEXT);
                return -1;
            };
            auto exps_of = [&](int32_t t, int32_t id) -> uint32_t {
                if (id < 0)
                    return 0x43434343u;          // (2^kShZeros)
                const int64_t at = (((int64_t)id * p.c.hkv + s.g) << p.c.page_shift) + ((t * kCkKeys + lane * 4) & in_page);
                return __ldg(reinterpret_cast<const uint32_t *>(exps + at));
            };
            // (page ids three tiles ahead, exponents two)
            int32_t id = checked(page_of(s.t0), s.t0), id1 = checked(page_of(s.t0 + 1), s.t0 + 1), id2 = page_of(s.t0 + 2);
            uint32_t e = exps_of(s.t0, id), e1 = exps_of(s.t0 + 1, id1);
            for (int32_t t = s.t0; t < s.t1; ++t, ++done) {
                id2 = checked(id2, t + 2);
                const int32_t id3 = page_of(t + 3);
                const uint32_t e2 = exps_of(t + 2, id2);
                int got = 1;
                if (lane == 0)
                    got = mbar_wait(bar_empty(slot), phase ^ 1u, abort_flag);
                if (!(ok = __shfl_sync(0xffffffffu, got, 0) != 0))
                    break;
                if (loads)
                    tma_load_4d_hint(sbase + p.off_ring + slot * Cfg::kRaw + lane * 4 * D, tm, bar_full(slot), 0, 0, s.g,
                                     id < 0 ? max(p.c.num_pages, 1) : id, pol);
                float f[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const uint32_t b = (e >> (8 * x)) & 0xffu;
                    f[x] = kv ? (float)(int8_t)(uint8_t)(b + 129u) : exp_byte_scale(b);   // b - 127, of 255 -128
                }
                st_shared_v4(sbase + p.off_raw + slot * 512 + lane * 16, __float_as_uint(f[0]), __float_as_uint(f[1]),
                             __float_as_uint(f[2]), __float_as_uint(f[3]));
                __syncwarp();
                if (lane == 0)
                    mbar_arrive_expect_tx(bar_full(slot), (uint32_t)Cfg::kRaw);
                __syncwarp();
                if ((slot += 2) >= nslot) {
                    slot -= nslot;
                    phase ^= 1u;
                }
                e = e1;
                e1 = e2;
                id = id1;
                id1 = id2;
                id2 = id3;
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
    } else {
        // ============================================================ computing warps
        const int q = lane & 3, r = lane >> 2;
        float *red = reinterpret_cast<float *>(smem);       // [8 warps][8 NB rows][D + 8]
        uint32_t slot = 0, phase = 0;
        bool ok = true;
        for (bool have = have0; have; have = ck_next<1>(p, s, v1)) {
            const int32_t nrows = s.ntok * p.G;
            // ---- Q: row r of each block in fp16, its largest magnitude at 2^14 or more, as operands; the
            // softmax factor (with the way back) and last visible key of rows 2 q and 2 q + 1
            uint32_t b0[NB][KS], b1[NB][KS];
            float c[NB][2];
            int32_t last[NB][2];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                const int32_t row0 = nb * 8, rho = row0 + r;
                const bool live = rho < nrows;
                const int32_t tok = live ? rho / p.G : 0, h = live ? rho - tok * p.G : 0;
                const uint2 *src = reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p.q) +
                                                                   (int64_t)(s.off + s.tb0 + tok) * p.q_stride +
                                                                   (int64_t)(s.g * p.G + h) * D + q * (D / 4));
                uint2 w[KS];
                uint32_t top = 0;
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    w[k] = live ? __ldg(src + k) : make_uint2(0u, 0u);
                    top = max(top, max(max(w[k].x & 0x7fffu, (w[k].x >> 16) & 0x7fffu),
                                       max(w[k].y & 0x7fffu, (w[k].y >> 16) & 0x7fffu)));
                }
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const int32_t shift = ck_q_shift(top);
                const float f = ck_pow2(shift), back = p.scale_log2 * ck_pow2(-shift);
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    b0[nb][k] = ck_pack_f16x2(bf16_lo(w[k].x) * f, bf16_hi(w[k].x) * f);
                    b1[nb][k] = ck_pack_f16x2(bf16_lo(w[k].y) * f, bf16_hi(w[k].y) * f);
                }
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    c[nb][x] = __shfl_sync(0xffffffffu, back, (2 * q + x) * 4);
                    const int32_t rx = row0 + 2 * q + x;
                    last[nb][x] = rx < nrows ? s.L + s.tb0 + rx / p.G : -1;
                }
            }
            float o[NB][NI / 2][4], mx[NB][2], l[NB][2], e_ref = 0.0f;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                mx[nb][0] = mx[nb][1] = -INFINITY;
                l[nb][0] = l[nb][1] = 0.0f;
#pragma unroll
                for (int i = 0; i < NI / 2; ++i)
                    o[nb][i][0] = o[nb][i][1] = o[nb][i][2] = o[nb][i][3] = 0.0f;
            }
            if (lane == 0)
                m->nan_at[warp] = INT32_MAX;
            __syncwarp();
            for (int32_t t = s.t0; t < s.t1 && ok; ++t) {
                const uint32_t vs = slot + 1;               // (slots come in pairs, nslot is even)
                ok = __all_sync(0xffffffffu, mbar_wait(bar_full(slot), phase, abort_flag) &&
                                                 mbar_wait(bar_full(vs), phase, abort_flag));
                if (!ok)
                    break;
                const int32_t k0 = t * kCkKeys;
                const bool masked = k0 + kCkKeys - 1 > s.L + s.tb0;
                const uint8_t *kt = smem + p.off_ring + slot * Cfg::kRaw, *vt = smem + p.off_ring + vs * Cfg::kRaw;
                const float *ke = reinterpret_cast<const float *>(smem + p.off_raw + slot * 512);
                const float *ve = reinterpret_cast<const float *>(smem + p.off_raw + vs * 512);
                const int kb = warp * 16;
                // ---- S^T of keys kb + r and kb + r + 8 with rows 2 q and 2 q + 1
                uint32_t w[2][KS];
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                    for (int h = 0; h < KS / 4; ++h) {
                        const uint4 x = *reinterpret_cast<const uint4 *>(
                            kt + sh_chunk<D>(kb + 8 * y + r, q * (KS / 4) + h));
                        w[y][4 * h] = x.x;
                        w[y][4 * h + 1] = x.y;
                        w[y][4 * h + 2] = x.z;
                        w[y][4 * h + 3] = x.w;
                    }
                float sc[NB][4];
                {
                    float s0[NB][4], s1[NB][4];     // two chains of products
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            s0[nb][x] = s1[nb][x] = 0.0f;
#pragma unroll
                    for (int k = 0; k < KS; ++k) {
                        uint32_t a0, a1, a2, a3;
                        sh_codes(w[0][k], a0, a2);
                        sh_codes(w[1][k], a1, a3);
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb)
                            sh_mma(k & 1 ? s1[nb] : s0[nb], a0, a1, a2, a3, b0[nb][k], b1[nb][k]);
                    }
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            sc[nb][x] = s0[nb][x] + s1[nb][x];
                }
                // ---- exponents and the running maximum
                const int key = kb + r;
                const float kf[2] = {ke[key], ke[key + 8]};
                float e[2] = {ve[key], ve[key + 8]};
                const bool low = fmaxf(e_ref - e[0], e_ref - e[1]) > kShSpan;
                float back[2] = {ck_pow2((int32_t)(e_ref - e[0])), ck_pow2((int32_t)(e_ref - e[1]))};
                uint32_t pb[NB][2];
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    float top[2];
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            float z = fmaf(sc[nb][2 * y + x], kf[y] * c[nb][x], e[y]);
                            if (masked)
                                z = k0 + key + 8 * y <= last[nb][x] ? z : -INFINITY;
                            sc[nb][2 * y + x] = z;
                        }
                        top[x] = fmaxf(sc[nb][x], sc[nb][2 + x]);
                    }
#pragma unroll
                    for (int w2 = 4; w2 < 32; w2 <<= 1) {
                        top[0] = fmaxf(top[0], __shfl_xor_sync(0xffffffffu, top[0], w2));
                        top[1] = fmaxf(top[1], __shfl_xor_sync(0xffffffffu, top[1], w2));
                    }
                    // (mx: the reference, the largest score less kCkLift when it last moved)
                    const bool up0 = top[0] > mx[nb][0] + (kCkSlack + kCkLift) || (mx[nb][0] == -INFINITY && top[0] != -INFINITY);
                    const bool up1 = top[1] > mx[nb][1] + (kCkSlack + kCkLift) || (mx[nb][1] == -INFINITY && top[1] != -INFINITY);
                    if (__any_sync(0xffffffffu, up0 || up1 || (nb == 0 && low))) {
                        if (nb == 0 && __any_sync(0xffffffffu, low)) {
                            // A row of zeros has e = kShZeros from here on: at the e = -112 with which it is written, P'
                            // would lose its weight beside rows of 2^10 or more.  A row whose byte stands for zeros becomes
                            // one; one of NaN counts as one, and where it lies is noted.  (A row past the last
                            // visible key may have any byte.)
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                const int32_t at = k0 + key + 8 * y;
                                const bool seen = at < s.len;
                                uint32_t some = 0;
#pragma unroll
                                for (int x = 0; x < D / 64; ++x) {
                                    const uint32_t chunk = sh_chunk<D>(key + 8 * y, q * (D / 64) + x);
                                    if (seen && e[y] <= kShZero) {
                                        st_shared_v4(smem_u32(vt) + chunk, 0u, 0u, 0u, 0u);
                                    } else {
                                        const uint4 w4 = *reinterpret_cast<const uint4 *>(vt + chunk);
                                        some |= (w4.x | w4.y | w4.z | w4.w) & 0x7f7f7f7fu;
                                    }
                                }
                                some |= __shfl_xor_sync(0xffffffffu, some, 1);
                                some |= __shfl_xor_sync(0xffffffffu, some, 2);
                                if (seen && e[y] <= kShZero) {
                                    if (e[y] == kShNan)
                                        atomicMin(&m->nan_at[warp], at);
                                    fence_proxy_async_smem();
                                }
                                if (!seen || some == 0u) {
                                    sc[0][2 * y] += kShZeros - e[y];
                                    sc[0][2 * y + 1] += kShZeros - e[y];
                                    e[y] = kShZeros;
                                }
                            }
#pragma unroll
                            for (int x = 0; x < 2; ++x) {
                                top[x] = fmaxf(sc[0][x], sc[0][2 + x]);
#pragma unroll
                                for (int w2 = 4; w2 < 32; w2 <<= 1)
                                    top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], w2));
                            }
                            const int32_t least = __reduce_min_sync(0xffffffffu, (int32_t)fminf(fminf(e[0], e[1]), 0.0f));
                            const float to = fminf(e_ref, (float)least + kShSpan), down = ck_pow2((int32_t)(to - e_ref));
                            e_ref = to;
                            back[0] = ck_pow2((int32_t)(e_ref - e[0]));
                            back[1] = ck_pow2((int32_t)(e_ref - e[1]));
#pragma unroll
                            for (int y = 0; y < NB; ++y) {
                                l[y][0] *= down;
                                l[y][1] *= down;
                            }
                            __syncwarp();
                        }
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const float mn = fmaxf(mx[nb][x], top[x] - kCkLift);
                            const float alpha = mx[nb][x] == -INFINITY ? 0.0f : fast_exp2(mx[nb][x] - mn);
                            mx[nb][x] = mn;
                            l[nb][x] *= alpha;
#pragma unroll
                            for (int i = 0; i < NI / 2; ++i) {
                                o[nb][i][x] *= alpha;
                                o[nb][i][2 + x] *= alpha;
                            }
                        }
                    }
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        float pr[2];
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const float mm = mx[nb][x] == -INFINITY ? 0.0f : mx[nb][x];
                            pr[x] = fast_exp2(sc[nb][2 * y + x] - mm);
                            l[nb][x] = fmaf(pr[x], back[y], l[nb][x]);
                        }
                        pb[nb][y] = sh_turn(ck_pack_f16x2(pr[0], pr[1]));   // row r, keys 8 y + 2 q, + 1
                    }
                }
                // ---- O^T += V^T P^T: keys kb + 2 q, + 1 and + 8, + 9 in a thread
                uint32_t v[4][NI / 4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int row = kb + 2 * q + (x & 1) + 8 * (x >> 1);
                    if constexpr (D == 128) {
                        const uint4 y = *reinterpret_cast<const uint4 *>(vt + sh_chunk<D>(row, r));
                        v[x][0] = y.x; v[x][1] = y.y; v[x][2] = y.z; v[x][3] = y.w;
                    } else {
                        const uint2 y = *reinterpret_cast<const uint2 *>(vt + sh_chunk<D>(row, r >> 1) + (r & 1) * 8);
                        v[x][0] = y.x; v[x][1] = y.y;
                    }
                    // (what lies past the last visible key may be NaN, which P' = 0 does not hide)
                    if (masked && k0 + row >= s.len) {
#pragma unroll
                        for (int j = 0; j < NI / 4; ++j)
                            v[x][j] = 0u;
                    }
                }
#pragma unroll
                for (int j = 0; j < NI / 4; ++j) {
                    uint32_t d[2][4];
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        // the codes of two keys side by side, one d after the other
                        sh_codes(__byte_perm(v[2 * x][j], v[2 * x + 1][j], 0x5140), d[x][0], d[x][1]);
                        sh_codes(__byte_perm(v[2 * x][j], v[2 * x + 1][j], 0x7362), d[x][2], d[x][3]);
                    }
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) {
                        sh_mma(o[nb][2 * j], d[0][0], d[0][1], d[1][0], d[1][1], pb[nb][0], pb[nb][1]);
                        sh_mma(o[nb][2 * j + 1], d[0][2], d[0][3], d[1][2], d[1][3], pb[nb][0], pb[nb][1]);
                    }
                }
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar_empty(slot));
                    mbar_arrive(bar_empty(vs));
                }
                if ((slot += 2) == nslot) {
                    slot = 0;
                    phase ^= 1u;
                }
            }
            // ---- join the warps: every warp's (m, l) and O, in units of 1 (NaN where the row sees a value row of
            // NaN), to shared memory, then four columns of a row a thread
            __syncwarp();
            const int32_t nan_at = m->nan_at[warp];
            const float o_scale = ck_pow2((int32_t)e_ref);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float z = l[nb][x];
#pragma unroll
                    for (int w2 = 4; w2 < 32; w2 <<= 1)
                        z += __shfl_xor_sync(0xffffffffu, z, w2);
                    const int row = nb * 8 + 2 * q + x;
                    if (r == 0)
                        m->ml[warp][row] = make_float2(mx[nb][x] - e_ref, z);
                    const float f = nan_at <= last[nb][x] ? NAN : o_scale;
                    // d = NI r + 2 i and + 1 at columns (2 i) 8 + r and (2 i + 1) 8 + r
                    float *dst = red + (warp * 8 * NB + row) * (D + 8) + r;
#pragma unroll
                    for (int i = 0; i < NI / 2; ++i) {
                        dst[16 * i] = o[nb][i][x] * f;
                        dst[16 * i + 8] = o[nb][i][2 + x] * f;
                    }
                }
            if (named_bar_any(1, 32 * kShWarps, !ok))
                break;                                      // (all eight warps leave together)
            const bool whole = s.t0 == 0 && s.t1 == s.nt;
            for (int32_t idx = tid; idx < nrows * (D / 4); idx += 32 * kShWarps) {
                const int32_t rho = idx / (D / 4), c4 = idx - rho * (D / 4);   // columns 4 c4 .. 4 c4 + 3
                const int32_t n = c4 / (NI / 4), i = (c4 - n * (NI / 4)) * 4;
                float M = -INFINITY;
                for (int32_t k = 0; k < kShWarps; ++k) {
                    const float2 x = m->ml[k][rho];
                    M = fmaxf(M, x.y != 0.0f ? x.x : -INFINITY);
                }
                float L = 0.0f, acc[4] = {0.f, 0.f, 0.f, 0.f};
                for (int32_t k = 0; k < kShWarps; ++k) {
                    const float2 x = m->ml[k][rho];
                    if (x.y == 0.0f)
                        continue;                           // no visible key: whatever its O holds
                    const float w = fast_exp2(x.x - M);
                    L += w * x.y;
                    const float *src = red + (k * 8 * NB + rho) * (D + 8) + i * 8 + n;
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        acc[y] = fmaf(w, src[8 * y], acc[y]);
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
                    const int64_t prow = (int64_t)(2 * cta + (s.t0 > 0 ? 0 : 1)) * kShortRows + rho;
                    *reinterpret_cast<float4 *>(p.part_o + prow * D + 4 * c4) = make_float4(acc[0], acc[1], acc[2], acc[3]);
                    if (c4 == 0)
                        p.part_ml[prow] = make_float2(M, L);
                }
            }
            if (!whole && s.t0 == 0 && tid == 0) {
                ChunkDesc d;
                d.np = ck_owner(shares, s.base + (int64_t)s.wt * (kStartKeys + (int64_t)kCkKeys * (s.nt - 1))) - cta + 1;
                d.row0 = s.off + s.tb0;
                d.ntok = s.ntok;
                d.g = s.g;
                p.desc[cta] = d;
            }
            named_bar_sync(1, 32 * kShWarps);               // the buffers are read
        }
    }
    __syncthreads();
    if (*abort_flag && tid == 0)
        set_status(p.status, SVP_DEV_TIMEOUT);
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
