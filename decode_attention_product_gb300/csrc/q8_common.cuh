// q8_common.cuh -- device helpers of the 8-bit block-scaled cache: the two code
// formats, their exact rounding and their widening.
//
// A block is one page (16 tokens) of one kv head's keys or values; its codes c
// stand for c * scale, scale one fp32 per block.
//   INT8   scale >= amax / 127, c = the integer nearest to x / scale
//   E4M3   scale = the least power of two with amax <= 448 * scale (a floating
//          code gains nothing from a finer scale, and x / scale is then exact,
//          so the hardware conversion is the only rounding)
// A code is the one nearest to the REAL quotient x / scale (ties to even), not
// to a rounded quotient: 32-bit division could land on a tie that is none.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace aq {

enum Q8Format { kInt8 = 0, kE4m3 = 1 };

// Nearest integer to x / s (ties to even), |x / s| <= 127.  q is off by at most
// one, and only near a half: the sign of x - (q +- 1/2) s decides, which one
// fused multiply-add gives exactly (q +- 1/2 has 8 bits).
__device__ __forceinline__ int nearest_int8(float x, float s, float inv) {
    const float q = rintf(x * inv);
    const float up = fmaf(-(q + 0.5f), s, x), dn = fmaf(-(q - 0.5f), s, x);
    int i = static_cast<int>(q);
    if (up > 0.f || (up == 0.f && (i & 1))) ++i;
    else if (dn < 0.f || (dn == 0.f && (i & 1))) --i;
    return i;
}

// Nearest integer to c * so / sn (ties to even), |c| <= 127, so <= sn: both
// products of the decision are split into a rounded part and its exact
// remainder, whose difference carries the exact sign.
__device__ __forceinline__ int rescale_int8(int c, float so, float sn, float ratio) {
    const float f = static_cast<float>(c);
    const float q = rintf(f * ratio);
    const float ph = f * so, pl = fmaf(f, so, -ph);
    auto side = [&](float mid) {
        const float mh = mid * sn, ml = fmaf(mid, sn, -mh);
        return (ph - mh) + (pl - ml);
    };
    const float up = side(q + 0.5f), dn = side(q - 0.5f);
    int i = static_cast<int>(q);
    if (up > 0.f || (up == 0.f && (i & 1))) ++i;
    else if (dn < 0.f || (dn == 0.f && (i & 1))) --i;
    return i;
}

__device__ __forceinline__ uint32_t e4m3x2_of(float lo, float hi) {
    return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ uint32_t h2_of_e4m3x2(uint32_t b) {
    const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(b & 0xffffu), __NV_E4M3);
    return static_cast<uint32_t>(r.x) | (static_cast<uint32_t>(r.y) << 16);
}

// Four INT8 codes as the halves 1152 + c - 1152: the byte c + 128 under the
// exponent of 1024 is 1024 + 128 + c, exact, and so is the difference.
__device__ __forceinline__ uint32_t h2_biased(uint32_t bytes) {        // bytes {b0, 0x64, b1, 0x64}
    const __half2 h = __hsub2(*reinterpret_cast<const __half2 *>(&bytes), __half2(__half_raw{0x6480}, __half_raw{0x6480}));
    return *reinterpret_cast<const uint32_t *>(&h);
}

// A word of four codes (dims d .. d + 3) as two fp16 pairs.
template <int FMT>
__device__ __forceinline__ void widen4(uint32_t w, uint32_t &lo, uint32_t &hi) {
    if (FMT == kInt8) {
        const uint32_t u = w ^ 0x80808080u;
        lo = h2_biased(__byte_perm(u, 0x64646464u, 0x4140));
        hi = h2_biased(__byte_perm(u, 0x64646464u, 0x4342));
    } else {
        lo = h2_of_e4m3x2(w);
        hi = h2_of_e4m3x2(w >> 16);
    }
}

// Four E4M3 codes as fp16 pairs of their values times 2^-8, by integer operations:
// sign, exponent and fraction moved to an fp16's places (subnormals stay exact; the
// codes are finite).
__device__ __forceinline__ void shift4_e4m3(uint32_t w, uint32_t &lo, uint32_t &hi) {
    const uint32_t top = ((w >> 1) & 0x3f3f3f3fu) | (w & 0x80808080u), low = (w << 7) & 0x80808080u;
    lo = __byte_perm(low, top, 0x5140);
    hi = __byte_perm(low, top, 0x7362);
}

// The scale of a block whose largest magnitude is `amax` (finite, >= 0).
template <int FMT>
__device__ __forceinline__ float scale_for(float amax) {
    if (!(amax > 0.f)) return 0.f;
    if (FMT == kInt8) return __fdiv_rn(amax, 127.0f);
    const uint32_t bits = __float_as_uint(amax);           // a normal float: amax >= 2^-24
    const uint32_t e = (bits >> 23) - ((bits & 0x7fffffu) <= 0x600000u ? 8u : 7u);   // 448 = 1.75 * 2^8
    return __uint_as_float(e << 23);
}

// What turns values into codes under one scale, worked out once per block.
// INT8: x * lo and x * hi, lo and hi a few units of 2^-24 below and above 1 / scale,
// are rounded to integers by the addition of 1.5 * 2^23 (one rounding, the code in
// the low byte).  x / scale lies between the two products: where they round alike
// the code is decided, else (a quotient within 2^-15 of a half) x is looked at
// exactly.  E4M3: x * lo is x / scale itself (a power of two).
struct Encoder {
    float scale, lo, hi;
    uint32_t keep;             // 0 where every code is 0 (scale 0 or NaN)
    bool all;                  // every value is looked at exactly (E4M3, a scale scale_for does not give)
};

template <int FMT>
__device__ __forceinline__ Encoder encoder_of(float scale) {
    Encoder e;
    const float inv = scale > 0.f ? __fdiv_rn(1.0f, scale) : 0.f;
    e.scale = scale;
    e.lo = FMT == kInt8 ? inv * (1.f - 0x1p-22f) : inv;
    e.hi = inv * (1.f + 0x1p-22f);
    e.keep = scale > 0.f ? 0xffffffffu : 0u;
    e.all = FMT == kE4m3 && scale > 0.f && (__float_as_uint(scale) & 0x7fffffu) != 0u;
    return e;
}

// Four values as codes; `again` where the exact decision has to be taken.
template <int FMT>
__device__ __forceinline__ uint32_t encode4(float4 x, const Encoder &e, bool &again) {
    if (FMT == kInt8) {
        auto round4 = [&](float inv) {
            constexpr float kMagic = 12582912.f;
            const uint32_t a = __float_as_uint(fmaf(x.x, inv, kMagic)), b = __float_as_uint(fmaf(x.y, inv, kMagic));
            const uint32_t c = __float_as_uint(fmaf(x.z, inv, kMagic)), d = __float_as_uint(fmaf(x.w, inv, kMagic));
            return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410) & e.keep;
        };
        const uint32_t w = round4(e.lo);
        again = w != round4(e.hi);
        return w;
    }
    again = e.all;
    return (e4m3x2_of(x.x * e.lo, x.y * e.lo) | (e4m3x2_of(x.z * e.lo, x.w * e.lo) << 16)) & e.keep;
}

template <int FMT>
__device__ __forceinline__ uint32_t encode4_exact(float4 x, float scale) {
    const float inv = __fdiv_rn(1.0f, scale);
    if (FMT == kInt8)
        return (static_cast<uint32_t>(nearest_int8(x.x, scale, inv)) & 0xffu) |
               ((static_cast<uint32_t>(nearest_int8(x.y, scale, inv)) & 0xffu) << 8) |
               ((static_cast<uint32_t>(nearest_int8(x.z, scale, inv)) & 0xffu) << 16) |
               (static_cast<uint32_t>(nearest_int8(x.w, scale, inv)) << 24);
    return e4m3x2_of(__fdiv_rn(x.x, scale), __fdiv_rn(x.y, scale)) |
           (e4m3x2_of(__fdiv_rn(x.z, scale), __fdiv_rn(x.w, scale)) << 16);
}

// Four codes of scale `from` rounded again under the larger scale `to`.
template <int FMT>
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float from, float to) {
    if (!(to > 0.f) || !(from > 0.f)) return 0u;
    const float ratio = __fdiv_rn(from, to);
    if (FMT == kInt8) {
        uint32_t r = 0u;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            r |= (static_cast<uint32_t>(
                      rescale_int8(static_cast<int8_t>((w >> (8 * j)) & 0xffu), from, to, ratio)) & 0xffu) << (8 * j);
        return r;
    }
    uint32_t lo, hi;
    widen4<FMT>(w, lo, hi);
    const float2 a = h2_to_f2(lo), b = h2_to_f2(hi);
    return e4m3x2_of(a.x * ratio, a.y * ratio) | (e4m3x2_of(b.x * ratio, b.y * ratio) << 16);
}

}  // namespace aq
