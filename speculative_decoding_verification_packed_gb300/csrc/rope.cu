// rope.cu -- rotary positions of a step's rows, alone or with the write of k and v into the pages.
//
// Pair t of a head turns by 2 pi pos f_t / 2^64, f_t in units of 2^-64 turns a position: the 64-bit
// product wraps at whole turns, so its upper 32 bits are the angle to 2^-32 of a turn at any position
// (an fp32 angle of position 10^6 would be 0.03 rad off).  Sine and cosine are fp32 (sincospif), so are
// the products; a row is rounded once, to its output's type or to the cache's.
//
// A block takes a few packed rows with all their heads: the rows' sines and cosines are made once, in
// shared memory, beside the lookup of their requests and pages; the first heads' data is on the way
// then.  A group of d / 8 lanes has every few heads of one row, eight elements a lane, so that a lane's
// sines and cosines stay in its registers from head to head (read from shared memory for each head they
// took as long as the rows: 21100 prompt rows of 48 heads x 128 then 180 us).  The other half of a pair
// (t, t + rot / 2) comes by a shuffle from rot / 16 lanes away, or, for a rot / 2 that is no multiple of 8,
// element by element from memory, with the sines read for every head (20000 such rows: 178 us with rot 36 or 18,
// where 48, 64 and 128 take 88 to 90).  All reads of a row come before its writes (one warp holds it), so
// an output may be its input.
//
// What bounds it: the chain cu -> context -> angle -> row for few rows (64 blocks of up to 16 rows, 11 MB: 5.0 us from
// a graph); memory for prompts (those 519 MB: 93 us, 5.6 TB/s), with the issue slots 57% busy beside it, so that
// occupancy counts: with 3 blocks an SM instead of 4, and four heads in flight instead of three, the
// blocks take 6.6 us.
#include <cmath>

#include "svp_cache.cuh"

namespace svp {

constexpr int kRopeThreads = 256;
constexpr int kRopeRows = 8;          // packed rows of a block, at most
template <int T> constexpr int kRopeAhead = T == SVP_F32 ? 2 : 3;   // heads of a group in flight

struct RopeParams {
    CacheParams c;
    const void *q, *k, *v;
    void *q_out, *k_out;
    int64_t q_stride, k_stride, qo_stride, ko_stride;   // elements
    const uint64_t *freq;
    const int32_t *pos, *ctx_len, *cu, *take;
    int32_t n, rows, hq, hkv, d, rot, inter, rpb;
    float scale;
    int32_t *status;
};

enum { kNoCache = -1 };

struct RopeRows {
    int64_t slot[kRopeRows], eoff[kRopeRows];   // place in the pools, -1: not written
    int32_t req[kRopeRows], at[kRopeRows];      // request (-1: row of none), cache position (-1: not written)
    int32_t ang[kRopeRows];                     // position for the angle
    float2 cs[kRopeRows][128];                  // scale (cos, sin) of pair t
};

// The block's rows: their requests, positions, places in the cache and angles.
template <int TC>
__device__ __forceinline__ void rope_rows(const RopeParams &p, int32_t r0, int32_t nr, RopeRows &m)
{
    const int tid = threadIdx.x;
    if (tid < kRopeRows)
        m.req[tid] = -1;
    __syncthreads();
    for (int32_t i = tid; i < p.n; i += kRopeThreads) {
        const int32_t off = __ldg(p.cu + i), end = __ldg(p.cu + i + 1);
        if (off < 0 || end < off || end > p.rows) {
            if (blockIdx.x == 0)
                set_status(p.status, SVP_DEV_BAD_SLOTS);
            continue;
        }
        const int32_t lo = max(off, r0), hi = min(end, r0 + nr);
        if (lo >= hi)
            continue;
        const int32_t first = p.ctx_len ? __ldg(p.ctx_len + i) : 0, k = end - off;
        int32_t took = k;
        if (TC != kNoCache && p.take)
            took = min(k, max(__ldg(p.take + i), 0));
        const bool fits = TC == kNoCache ? (int64_t)first + k <= ((int64_t)1 << 31)
                                         : took == 0 || (int64_t)first + took <= ((int64_t)p.c.max_pages << p.c.page_shift);
        if ((TC != kNoCache || !p.pos) && ((first < 0 && took > 0) || !fits)) {
            set_status(p.status, SVP_DEV_BAD_CONTEXT);
            continue;
        }
        for (int32_t r = lo; r < hi; ++r) {
            m.req[r - r0] = i;
            // (rows behind take have a position for their angle, which wraps as an int32 does)
            m.ang[r - r0] = p.pos ? __ldg(p.pos + r) : (int32_t)((uint32_t)first + (uint32_t)(r - off));
            m.at[r - r0] = TC != kNoCache && r - off < took ? first + (r - off) : -1;
        }
    }
    __syncthreads();
    if (TC != kNoCache && tid < nr) {
        const int32_t i = m.req[tid], at = m.at[tid];
        int64_t slot = -1, eoff = 0;
        if (i >= 0 && at >= 0) {
            const int32_t page = __ldg(p.c.block_table + (int64_t)i * p.c.max_pages + (at >> p.c.page_shift));
            const int32_t tok = at & ((1 << p.c.page_shift) - 1);
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
    const int32_t pairs = p.rot >> 1;
    for (int32_t x = tid; x < nr * pairs; x += kRopeThreads) {
        const int32_t r = x / pairs, t = x - r * pairs;
        if (m.req[r] < 0)
            continue;
        const uint64_t turn = (uint64_t)(int64_t)m.ang[r] * __ldg(p.freq + t);
        float s, c;
        sincospif((float)(int32_t)(turn >> 32) * 4.656612873077393e-10f, &s, &c);   // half turns: 2^-31
        m.cs[r][t] = make_float2(c * p.scale, s * p.scale);
    }
    __syncthreads();
}

// One element of a pair, x cos + y (-sin, or sin for the second one): the same operations wherever it is made.
__device__ __forceinline__ float rope_turn(float x, float y, float c, float s) { return fmaf(x, c, __fmul_rn(y, s)); }

__device__ __forceinline__ uint64_t rope_mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

template <int T>
__device__ __forceinline__ float rope_one(const void *base, int64_t e)
{
    if constexpr (T == SVP_F32)
        return static_cast<const float *>(base)[e];
    else
        return __uint_as_float((uint32_t)static_cast<const uint16_t *>(base)[e] << 16);
}

// Eight elements of a row in storage, as words.
template <int T> constexpr int kRopeWords = kWords<T> / 2;

template <int T>
__device__ __forceinline__ void rope_load(const void *base, int64_t e, uint32_t (&w)[kRopeWords<T>])
{
    const uint4 *s = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(base) + e * (kWords<T> / 4));
#pragma unroll
    for (int i = 0; i < kRopeWords<T> / 4; ++i) {
        const uint4 v = s[i];
        w[4 * i] = v.x;
        w[4 * i + 1] = v.y;
        w[4 * i + 2] = v.z;
        w[4 * i + 3] = v.w;
    }
}

template <int T>
__device__ __forceinline__ void rope_store(void *base, int64_t e, const uint32_t (&w)[kRopeWords<T>])
{
    uint8_t *at = static_cast<uint8_t *>(base) + e * (kWords<T> / 4);
    if constexpr (T == SVP_E4M3) {
        *reinterpret_cast<uint2 *>(at) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
        for (int i = 0; i < kRopeWords<T> / 4; ++i)
            reinterpret_cast<uint4 *>(at)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
}

template <int T>
__device__ __forceinline__ void rope_widen(const uint32_t (&w)[kRopeWords<T>], float (&x)[8])
{
#pragma unroll
    for (int i = 0; i < kRopeWords<T>; ++i) {
        if constexpr (T == SVP_F32) {
            x[i] = __uint_as_float(w[i]);
        } else {
            x[2 * i] = bf16_lo(w[i]);
            x[2 * i + 1] = bf16_hi(w[i]);
        }
    }
}

template <int T>
__device__ __forceinline__ void rope_narrow(const float (&x)[8], uint32_t (&w)[kRopeWords<T>])
{
#pragma unroll
    for (int i = 0; i < kRopeWords<T>; ++i)
        w[i] = T == SVP_F32 ? __float_as_uint(x[i]) : pack_bf16x2(x[2 * i], x[2 * i + 1]);
}

// TIn: type of the rows; TC: of the cache, or kNoCache (k goes to k_out).
template <int TIn, int TC>
__global__ void __launch_bounds__(kRopeThreads, 4) rope_kernel(const __grid_constant__ RopeParams p)
{
    constexpr int A = kRopeAhead<TIn>;
    __shared__ RopeRows m;
    griddep_launch_dependents();
    griddep_wait();
    const int32_t r0 = (int32_t)blockIdx.x * p.rpb;
    const int32_t nr = min(p.rpb, p.rows - r0), hq = p.hq, hkv = p.hkv;
    const int32_t cols = hq + (TC == kNoCache ? 1 : 2) * hkv;
    const int gl = p.d >> 3, half = p.rot >> 1;
    const int grp = threadIdx.x / gl, lane = threadIdx.x - grp * gl;
    // groups g, g + rpb, .. have row g (rpb divides their number), `step` of them
    const int32_t step = kRopeThreads / gl / p.rpb, r = grp % p.rpb, first = grp / p.rpb;
    const int32_t turns = (cols + step - 1) / step;       // heads of a group
    const int e0 = lane * 8;
    uint32_t raw[A][kRopeWords<TIn>];
    // column c (a head of q, then of k, then of v) of this row is at source(c) + c * d
    constexpr int kSize = TIn == SVP_F32 ? 4 : 2;
    const int32_t hd = p.d * kSize;
    const uint8_t *const in_q = static_cast<const uint8_t *>(p.q) + (r0 + r) * p.q_stride * kSize;
    const uint8_t *const in_k = static_cast<const uint8_t *>(p.k) + ((r0 + r) * p.k_stride - (int64_t)hq * p.d) * kSize;
    const uint8_t *const in_v =
        TC == kNoCache ? nullptr : static_cast<const uint8_t *>(p.v) + ((r0 + r) * p.k_stride - (int64_t)(hq + hkv) * p.d) * kSize;
    uint8_t *const out_q = static_cast<uint8_t *>(p.q_out) + (r0 + r) * p.qo_stride * kSize + e0 * kSize;
    uint8_t *const out_k =
        TC != kNoCache ? nullptr : static_cast<uint8_t *>(p.k_out) + ((r0 + r) * p.ko_stride - (int64_t)hq * p.d) * kSize + e0 * kSize;
    auto source = [&](int32_t c) -> const uint8_t * {
        return (c < hq ? in_q : TC == kNoCache || c < hq + hkv ? in_k : in_v) + (int64_t)c * hd;
    };
    auto fetch = [&](int32_t turn, uint32_t (&w)[kRopeWords<TIn>]) {
        const int32_t c = first + turn * step;
        if (r < nr && c < cols)
            rope_load<TIn>(source(c), e0, w);
    };
#pragma unroll
    for (int u = 0; u < A; ++u)
        fetch(u, raw[u]);
    rope_rows<TC>(p, r0, nr, m);
    const bool live = r < nr && m.req[r < nr ? r : 0] >= 0;
    const int64_t slot0 = TC != kNoCache && live ? m.slot[r] : -1;
    // this lane's sines and cosines.  Pairs (t, t + half) by eights: its elements are all first ones of their pairs,
    // all second ones, or beyond rot
    const bool eights = !p.inter && (half & 7) == 0, second = e0 >= half;
    const bool mine = p.inter ? lane * 4 < half : e0 < p.rot;
    float2 cs[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        cs[i] = make_float2(1.0f, 0.0f);
    if (live && mine && (p.inter || eights)) {
        const float2 *at = m.cs[r] + (p.inter ? lane * 4 : e0 - (second ? half : 0));
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (p.inter ? i < 4 && lane * 4 + i < half : true)
                cs[i] = at[i];
        if (eights && !second) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                cs[i].y = -cs[i].y;
        }
    }
    const int there = (threadIdx.x & 31) + (!mine ? 0 : second ? -(half >> 3) : half >> 3);
    // every thread of the block runs every turn: the shuffles are over whole warps
    for (int32_t t0 = 0; t0 < turns; t0 += A) {
#pragma unroll
        for (int u = 0; u < A; ++u) {
            const int32_t c = first + (t0 + u) * step;
            const bool have = live && c < cols, turn = have && c < hq + hkv;
            float x[8];
            if (have)
                rope_widen<TIn>(raw[u], x);
            if (p.inter) {
                if (turn && mine) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (lane * 4 + i < half) {
                            const float a = x[2 * i], b = x[2 * i + 1];
                            x[2 * i] = rope_turn(a, b, cs[i].x, -cs[i].y);
                            x[2 * i + 1] = rope_turn(b, a, cs[i].x, cs[i].y);
                        }
                    }
                }
            } else if (eights) {
                float y[8];
                uint32_t other[kRopeWords<TIn>];
#pragma unroll
                for (int i = 0; i < kRopeWords<TIn>; ++i)
                    other[i] = __shfl_sync(0xffffffffu, raw[u][i], there);
                rope_widen<TIn>(other, y);
                if (turn && mine) {
#pragma unroll
                    for (int i = 0; i < 8; i += 2)
                        f32x2_unpack(f32x2_fma(f32x2_pack(x[i], x[i + 1]), f32x2_pack(cs[i].x, cs[i + 1].x),
                                               rope_mul2(f32x2_pack(y[i], y[i + 1]), f32x2_pack(cs[i].y, cs[i + 1].y))),
                                     x[i], x[i + 1]);
                }
            } else if (turn && mine) {
                const uint8_t *base = source(c);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int e = e0 + i;
                    if (e < p.rot) {
                        const bool late = e >= half;
                        const float y = rope_one<TIn>(base, late ? e - half : e + half);
                        const float2 w = m.cs[r][late ? e - half : e];
                        x[i] = rope_turn(x[i], y, w.x, late ? w.y : -w.y);
                    }
                }
            }
            __syncwarp();                                 // (the row has been read: its output may lie over it)
            if (have && (c < hq || TC == kNoCache)) {
                uint32_t w[kRopeWords<TIn>];
                rope_narrow<TIn>(x, w);
                rope_store<TIn>((TC != kNoCache || c < hq ? out_q : out_k) + (int64_t)c * hd, 0, w);
            }
            if constexpr (TC != kNoCache) {
                const bool v = c >= hq + hkv;
                const bool store = have && c >= hq && slot0 >= 0;
                const int32_t h = c - hq - (v ? hkv : 0);
                const int64_t e = slot0 + h * p.c.s_head + e0;
                void *pool = v ? p.c.v : p.c.k;
                if constexpr (TC == SVP_E4M3) {
                    uint32_t amax = 0u;
                    if (store) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            amax = max(amax, __float_as_uint(x[i]) & 0x7fffffffu);
                    }
                    for (int o = gl >> 1; o > 0; o >>= 1)
                        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                    if (store) {
                        const bool fine = amax < 0x7f800000u;
                        const uint32_t b = fine ? exp_byte_of(amax) : 255u;
                        const float inv = __uint_as_float((254u - b) << 23);   // 2^-(b - 127)
                        uint32_t w[2] = {0u, 0u};
                        if (fine) {
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                w[i] = pack_e4m3x2(x[4 * i] * inv, x[4 * i + 1] * inv) |
                                       (pack_e4m3x2(x[4 * i + 2] * inv, x[4 * i + 3] * inv) << 16);
                        }
                        rope_store<SVP_E4M3>(pool, e, w);
                        if (lane == 0)
                            (v ? p.c.v_exp : p.c.k_exp)[m.eoff[r] + ((int64_t)h << p.c.page_shift)] = (uint8_t)b;
                    }
                } else if (store) {
                    if (TIn == TC && v) {
                        if constexpr (TIn == TC)
                            rope_store<TC>(pool, e, raw[u]);              // bits as they are
                    } else {
                        uint32_t w[kRopeWords<TC>];
                        rope_narrow<TC>(x, w);
                        rope_store<TC>(pool, e, w);
                    }
                }
            }
            fetch(t0 + u + A, raw[u]);
        }
    }
}

int sm_count();

template <int TIn, int TC>
static svp_status rope_launch(RopeParams &p, cudaStream_t stream)
{
    // one row a block while that leaves fewer than four blocks an SM, then a power of two (each row has as many groups
    // of lanes; 8 at d = 256, where a block has eight)
    const int32_t want = p.rows / (4 * sm_count());
    p.rpb = 1;
    while (p.rpb * 2 <= want && p.rpb < kRopeRows)
        p.rpb *= 2;
    const unsigned grid = (unsigned)((p.rows + p.rpb - 1) / p.rpb);
    return launch_pdl(rope_kernel<TIn, TC>, dim3(grid), dim3(kRopeThreads), 0, stream, p) == cudaSuccess ? SVP_OK
                                                                                                         : SVP_ECUDA;
}

static bool al16(const void *x) { return (reinterpret_cast<uintptr_t>(x) & 15) == 0; }

static svp_status rope_common(RopeParams &p, const svp_rotary *rotary, svp_dtype dtype, int32_t n, int32_t m_cap, int32_t d)
{
    if (!rotary || n < 0 || m_cap < 0)
        return SVP_EINVAL;
    if (d != 64 && d != 128 && d != 256)
        return SVP_EUNSUPPORTED;
    if (dtype != SVP_F32 && dtype != SVP_BF16)
        return SVP_EUNSUPPORTED;
    if (rotary->rot < 2 || rotary->rot > d || (rotary->rot & 1) || !std::isfinite(rotary->scale) ||
        (rotary->interleaved != 0 && rotary->interleaved != 1))
        return SVP_EINVAL;
    p.freq = rotary->freq;
    p.rot = rotary->rot;
    p.inter = rotary->interleaved;
    p.scale = rotary->scale;
    p.n = n;
    p.rows = m_cap;
    p.d = d;
    return SVP_OK;
}

static bool rope_stride(int64_t stride, int32_t heads, int32_t d, svp_dtype dtype)
{
    return heads > 0 && stride >= (int64_t)heads * d && (stride * (dtype == SVP_F32 ? 4 : 2)) % 16 == 0;
}

}  // namespace svp

using namespace svp;

extern "C" {

svp_status svp_rope_frequencies(int32_t rot, double base, svp_rope_scaling scaling, double factor, int32_t original,
                                double slow, double fast, uint64_t *freq)
{
    if (!freq || rot < 2 || (rot & 1) || !(base > 1.0) || !std::isfinite(base) || !(factor > 0.0) || !std::isfinite(factor))
        return SVP_EINVAL;
    if (scaling != SVP_ROPE_NONE && scaling != SVP_ROPE_LINEAR && scaling != SVP_ROPE_NTK && scaling != SVP_ROPE_YARN)
        return SVP_EUNSUPPORTED;
    if (scaling == SVP_ROPE_YARN && (original < 1 || !(slow > 0.0) || !(fast > slow) || !std::isfinite(fast)))
        return SVP_EINVAL;
    const double two_pi = 6.283185307179586476925286766559;
    if (scaling == SVP_ROPE_NTK && rot > 2)
        base *= std::pow(factor, (double)rot / (rot - 2));
    double lo = 0.0, hi = 0.0;
    if (scaling == SVP_ROPE_YARN) {
        // pair t turns original * base^(-2t / rot) / 2 pi times in the original length
        const auto pair_of = [&](double turns) { return rot * std::log(original / (turns * two_pi)) / (2.0 * std::log(base)); };
        lo = std::fmax(std::floor(pair_of(fast)), 0.0);
        hi = std::fmin(std::ceil(pair_of(slow)), (double)rot - 1.0);
    }
    for (int32_t t = 0; t < rot / 2; ++t) {
        double f = std::pow(base, -2.0 * t / rot);
        if (scaling == SVP_ROPE_LINEAR)
            f /= factor;
        if (scaling == SVP_ROPE_YARN) {
            const double ramp = std::fmin(std::fmax((t - lo) / std::fmax(hi - lo, 0.001), 0.0), 1.0);
            f = f * (1.0 - ramp) + f / factor * ramp;
        }
        const double turns = f / two_pi, part = turns - std::floor(turns);
        const double units = std::ldexp(part, 64);        // (exact; below 2^64)
        freq[t] = units >= 18446744073709551616.0 ? 0u : (uint64_t)units;
    }
    return SVP_OK;
}

svp_status svp_rope(const void *q, int64_t q_row_stride, const void *k, int64_t k_row_stride, svp_dtype dtype,
                    const svp_rotary *rotary, const int32_t *pos, const int32_t *ctx_len, const int32_t *cu_slots,
                    int32_t n, int32_t m_cap, int32_t hq, int32_t hkv, int32_t d, void *q_out, int64_t q_out_stride,
                    void *k_out, int64_t k_out_stride, void *ws, size_t ws_bytes, void *stream)
{
    RopeParams p{};
    const svp_status st = rope_common(p, rotary, dtype, n, m_cap, d);
    if (st != SVP_OK)
        return st;
    if (!q == !!q_out || !k == !!k_out)
        return SVP_EINVAL;
    if (q && (!rope_stride(q_row_stride, hq, d, dtype) || !rope_stride(q_out_stride, hq, d, dtype)))
        return SVP_EINVAL;
    if (k && (!rope_stride(k_row_stride, hkv, d, dtype) || !rope_stride(k_out_stride, hkv, d, dtype)))
        return SVP_EINVAL;
    if ((q && q == q_out && q_row_stride != q_out_stride) || (k && k == k_out && k_row_stride != k_out_stride))
        return SVP_EINVAL;
    if (!ws || ws_bytes < kWsHeader)
        return SVP_EWORKSPACE;
    if (n == 0 || m_cap == 0 || (!q && !k))
        return SVP_OK;
    if (!p.freq || !cu_slots || (!ctx_len && !pos) || !al16(q) || !al16(k) || !al16(q_out) || !al16(k_out))
        return SVP_EINVAL;
    p.q = q;
    p.k = k;
    p.q_out = q_out;
    p.k_out = k_out;
    p.q_stride = q_row_stride;
    p.k_stride = k_row_stride;
    p.qo_stride = q_out_stride;
    p.ko_stride = k_out_stride;
    p.pos = pos;
    p.ctx_len = ctx_len;
    p.cu = cu_slots;
    p.hq = q ? hq : 0;
    p.hkv = k ? hkv : 0;
    p.status = static_cast<int32_t *>(ws);
    return dtype == SVP_F32 ? rope_launch<SVP_F32, kNoCache>(p, (cudaStream_t)stream)
                            : rope_launch<SVP_BF16, kNoCache>(p, (cudaStream_t)stream);
}

svp_status svp_rope_cache_write(const void *q, int64_t q_row_stride, const void *k, const void *v, int64_t kv_row_stride,
                                svp_dtype dtype, const svp_rotary *rotary, const svp_cache *cache, const int32_t *pos,
                                const int32_t *ctx_len, const int32_t *cu_slots, const int32_t *take, int32_t n,
                                int32_t m_cap, int32_t hq, int32_t hkv, int32_t d, void *q_out, int64_t q_out_stride,
                                void *ws, size_t ws_bytes, void *stream)
{
    RopeParams p{};
    svp_status st = rope_common(p, rotary, dtype, n, m_cap, d);
    if (st != SVP_OK)
        return st;
    st = cache_params(cache, hkv, d, p.c);
    if (st != SVP_OK)
        return st;
    if (!q == !!q_out || (q && q == q_out && q_row_stride != q_out_stride))
        return SVP_EINVAL;
    if (q && (!rope_stride(q_row_stride, hq, d, dtype) || !rope_stride(q_out_stride, hq, d, dtype)))
        return SVP_EINVAL;
    if (!rope_stride(kv_row_stride, hkv, d, dtype))
        return SVP_EINVAL;
    if (!ws || ws_bytes < kWsHeader)
        return SVP_EWORKSPACE;
    if (n == 0 || m_cap == 0)
        return SVP_OK;
    if (!p.freq || !k || !v || !ctx_len || !cu_slots || !al16(q) || !al16(k) || !al16(v) || !al16(q_out))
        return SVP_EINVAL;
    p.q = q;
    p.k = k;
    p.v = v;
    p.q_out = q_out;
    p.q_stride = q_row_stride;
    p.k_stride = kv_row_stride;
    p.qo_stride = q_out_stride;
    p.pos = pos;
    p.ctx_len = ctx_len;
    p.cu = cu_slots;
    p.take = take;
    p.hq = q ? hq : 0;
    p.hkv = hkv;
    p.status = static_cast<int32_t *>(ws);
    cudaStream_t s = (cudaStream_t)stream;
    if (dtype == SVP_F32) {
        switch (cache->dtype) {
        case SVP_F32: return rope_launch<SVP_F32, SVP_F32>(p, s);
        case SVP_BF16: return rope_launch<SVP_F32, SVP_BF16>(p, s);
        default: return rope_launch<SVP_F32, SVP_E4M3>(p, s);
        }
    }
    switch (cache->dtype) {
    case SVP_F32: return rope_launch<SVP_BF16, SVP_F32>(p, s);
    case SVP_BF16: return rope_launch<SVP_BF16, SVP_BF16>(p, s);
    default: return rope_launch<SVP_BF16, SVP_E4M3>(p, s);
    }
}

}  // extern "C"
