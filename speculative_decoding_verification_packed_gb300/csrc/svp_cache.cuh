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

// Four e4m3 codes (bytes 0..3 of w) as fp32: the byte's sign, exponent and mantissa fields are
// put at those of a bf16 number, which is the code's value times 2^-120 (e4m3 subnormals become
// bf16 subnormals), and the product with 2^120 is exact.
__device__ __forceinline__ void e4m3x4_to_f32(uint32_t w, float (&f)[4])
{
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t b = (w >> (8 * e)) & 0xffu;
        f[e] = __uint_as_float(((b & 0x80u) << 24) | ((b & 0x7fu) << 20)) * 0x1p120f;
    }
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

}  // namespace svp
