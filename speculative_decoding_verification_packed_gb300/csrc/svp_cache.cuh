// svp_cache.cuh -- the paged cache as the kernels see it: pools, block table, 8-bit rows.
#pragma once

#include "svp_device.cuh"

namespace svp {

struct CacheParams {
    void *k, *v;
    uint8_t *k_exp, *v_exp;
    const int32_t *block_table;
    int64_t s_page, s_head, s_tok;   // element strides of the pools
    int32_t max_pages, page_shift, num_pages, hkv;
};

// Host checks shared by the cache's calls; fills cp.  SVP_OK, SVP_EINVAL or SVP_EUNSUPPORTED.
svp_status cache_params(const svp_cache *cache, int32_t hkv, int32_t d, CacheParams &cp);

// 2^(b - 127) of an exponent byte; 255 stands for NaN (and 0 for 0).
__device__ __forceinline__ float exp_byte_scale(uint32_t b)
{
    return __uint_as_float(b == 255u ? 0x7fc00000u : b << 23);
}

// Four e4m3 codes (bytes 0..3 of w) as fp32 (through fp16, which holds every code).
__device__ __forceinline__ void e4m3x4_to_f32(uint32_t w, float (&f)[4])
{
    asm("{\n\t.reg .b16 a, b, c, d;\n\t.reg .b32 x;\n\t"
        "mov.b32 {a, b}, %4;\n\t"
        "cvt.rn.f16x2.e4m3x2 x, a;\n\t"
        "mov.b32 {c, d}, x;\n\t"
        "cvt.f32.f16 %0, c;\n\t"
        "cvt.f32.f16 %1, d;\n\t"
        "cvt.rn.f16x2.e4m3x2 x, b;\n\t"
        "mov.b32 {c, d}, x;\n\t"
        "cvt.f32.f16 %2, c;\n\t"
        "cvt.f32.f16 %3, d;\n\t}"
        : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3])
        : "r"(w));
}

// Byte of the smallest power of two that takes magnitude bits `amax` (fp32, finite) to 448 =
// 1.75 * 2^8 or less: with amax = 1.f * 2^(E - 127) that is 2^(E - 135), one more when 1.f > 1.75.
__device__ __forceinline__ uint32_t exp_byte_of(uint32_t amax)
{
    const int32_t b = (int32_t)(amax >> 23) - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);
    return (uint32_t)(b < 15 ? 15 : b);
}

// Two fp32 values (|x| <= 448) to e4m3, nearest even; the low byte holds `lo`.
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Sixteen elements of a row in storage, as words.
template <int T> constexpr int kWords = T == SVP_F32 ? 16 : T == SVP_BF16 ? 8 : 4;

template <int T>
__device__ __forceinline__ void load16(const void *base, int64_t e, uint32_t (&w)[kWords<T>])
{
    const uint4 *s = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(base) + e * (kWords<T> / 4));
#pragma unroll
    for (int i = 0; i < kWords<T> / 4; ++i) {
        const uint4 v = s[i];
        w[4 * i] = v.x;
        w[4 * i + 1] = v.y;
        w[4 * i + 2] = v.z;
        w[4 * i + 3] = v.w;
    }
}

template <int T>
__device__ __forceinline__ void store16(void *base, int64_t e, const uint32_t (&w)[kWords<T>])
{
    uint4 *s = reinterpret_cast<uint4 *>(static_cast<uint8_t *>(base) + e * (kWords<T> / 4));
#pragma unroll
    for (int i = 0; i < kWords<T> / 4; ++i)
        s[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
}

template <int T>
__device__ __forceinline__ void to_f32(const uint32_t (&w)[kWords<T>], float (&x)[16])
{
#pragma unroll
    for (int i = 0; i < kWords<T>; ++i) {
        if constexpr (T == SVP_F32) {
            x[i] = __uint_as_float(w[i]);
        } else if constexpr (T == SVP_BF16) {
            x[2 * i] = bf16_lo(w[i]);
            x[2 * i + 1] = bf16_hi(w[i]);
        } else {
            float f[4];
            e4m3x4_to_f32(w[i], f);
#pragma unroll
            for (int y = 0; y < 4; ++y)
                x[4 * i + y] = f[y];
        }
    }
}

template <int T>
__device__ __forceinline__ void from_f32(const float (&x)[16], uint32_t (&w)[kWords<T>])
{
    static_assert(T != SVP_E4M3, "8-bit rows are made with their exponent byte");
#pragma unroll
    for (int i = 0; i < kWords<T>; ++i)
        w[i] = T == SVP_F32 ? __float_as_uint(x[i]) : pack_bf16x2(x[2 * i], x[2 * i + 1]);
}

// Bits of the largest magnitude (as fp32) of sixteen elements.
template <int T>
__device__ __forceinline__ uint32_t amax16(const uint32_t (&w)[kWords<T>])
{
    uint32_t m = 0u;
    if constexpr (T == SVP_F32) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            m = max(m, w[i] & 0x7fffffffu);
        return m;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            m = __vmaxu2(m, w[i] & 0x7fff7fffu);
        return max(m & 0xffff0000u, m << 16);
    }
}

}  // namespace svp
