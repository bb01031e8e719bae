// The 8-bit form of an activation row: e4m3 codes and one power-of-two exponent per 32 values.
//
// For each 32 neighbouring values, e is the smallest exponent that brings the largest finite |x|
// to at most 448 (e4m3's largest value): |x| <= 448 * 2^e. The code is x * 2^-e rounded to nearest
// even; a power of two makes that multiplication exact, so the only rounding is e4m3's own (2^-4
// relative for |x| >= 2^(e-6), 2^(e-10) absolute below) and nothing saturates. e + 127 is kept in
// a byte (0 for a block without a nonzero finite value). An infinity or NaN becomes NaN.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cstdint>

namespace lowbit {

__device__ __forceinline__ uint32_t finite_abs_bf16(uint32_t h) {   // 0 for infinities and NaN
    h &= 0x7FFFu;
    return h >= 0x7F80u ? 0u : h;
}

// Exponent byte of a block from the bits of its largest finite |x| (bf16). Subnormal bf16 values
// give an exponent below -127 + 0 either way: the byte is clamped at 0.
__device__ __forceinline__ uint32_t checkpoint_exponent(uint32_t amax) {
    // |x| = m * 2^(E - 127), m in [1, 2): 448 = 1.75 * 2^8, so e = E - 127 - 8 (+ 1 if m > 1.75)
    const int e = static_cast<int>(amax >> 7) - 8 + ((amax & 0x7Fu) > 0x60u ? 1 : 0);
    return amax == 0 ? 0u : static_cast<uint32_t>(max(0, e));
}

// Eight bf16 values of one thread -> eight codes; the block's four neighbouring lanes (aligned to 4)
// call together. `exponent` is the block's byte. The product with 2^-e is formed in bf16 (exact, or
// below e4m3's range); a block with an infinity or NaN takes the longer way.
__device__ __forceinline__ uint2 checkpoint_encode8(const uint4& v, uint8_t& exponent) {
    uint32_t in[4] = {v.x, v.y, v.z, v.w};
    auto lanes_max = [](uint32_t m) {
        m = max(m & 0xFFFFu, m >> 16);
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        return max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    };
    constexpr uint32_t kAbs = 0x7FFF7FFFu;
    uint32_t m = lanes_max(__vmaxs2(__vmaxs2(in[0] & kAbs, in[1] & kAbs), __vmaxs2(in[2] & kAbs, in[3] & kAbs)));
    if (__any_sync(0xffffffffu, m >= 0x7F80u)) {
        uint32_t f = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f = max(f, max(finite_abs_bf16(in[i]), finite_abs_bf16(in[i] >> 16)));
            if ((in[i] & 0x7F80u) == 0x7F80u) in[i] |= 0x7FFFu;               // an infinity becomes NaN too
            if ((in[i] & 0x7F800000u) == 0x7F800000u) in[i] |= 0x7FFF0000u;
        }
        m = lanes_max(f);
    }
    const uint32_t kept = checkpoint_exponent(m);
    exponent = static_cast<uint8_t>(kept);
    // 2^(127 - kept): kept <= 247, so the scale is a normal number
    const uint32_t s1 = (254u - kept) << 7, s2 = s1 | (s1 << 16);
    uint32_t pair[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&in[i]),
                                         *reinterpret_cast<const __nv_bfloat162*>(&s2));
        const uint32_t w = *reinterpret_cast<const uint32_t*>(&y);
        pair[i] = __nv_cvt_float2_to_fp8x2(make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)),
                                           __NV_SATFINITE, __NV_E4M3);
    }
    return make_uint2(__byte_perm(pair[0], pair[1], 0x5410), __byte_perm(pair[2], pair[3], 0x5410));
}

// Eight codes -> eight bf16 values (two per word). Exact: four significant bits times a power of
// two (below bf16's smallest subnormal the product rounds).
__device__ __forceinline__ uint4 checkpoint_decode8(const uint2& c, uint32_t exponent) {
    const float scale = exponent ? __uint_as_float(exponent << 23) : __uint_as_float(0x00400000u);   // 2^(exponent - 127)
    uint32_t out[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t two = ((i < 2 ? c.x : c.y) >> (16 * (i & 1))) & 0xFFFFu;
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two), __NV_E4M3);
        const float2 f = __half22float2(__half2(h));
        const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * scale, f.y * scale);
        out[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(out[0], out[1], out[2], out[3]);
}

}  // namespace lowbit
