// fp8_device.hpp - E4M3 quantization helpers shared by the per-row and the per-block FP8 quantizers.
#pragma once

#include "mx_device.hpp"

namespace mx {

// fl32(x / s) for BF16 rows: r = fl32(1 / s) once per row, then the quotient q0 = fl32(x r) is
// corrected twice with the remainder x - q s (exact, an FMA) scaled by r (Markstein's method); the
// sign of x is restored for zeros.  Used only when s >= 2^-90, so that every remainder that can
// decide a code is a normal number.  An exhaustive comparison with the IEEE division, over every
// finite positive BF16 row maximum a (s = fl32(a / 448) >= 2^-90) and every BF16 x with |x| <= a,
// found the same quotient wherever it is at least 2^-10 (below that every code is a signed zero)
// and the same E4M3 code everywhere.
__device__ __forceinline__ float div_corrected(float x, float s, float r) {
    const float q0 = x * r;
    const float q1 = __builtin_fmaf(__builtin_fmaf(-q0, s, x), r, q0);
    const float q2 = __builtin_fmaf(__builtin_fmaf(-q1, s, x), r, q1);
    return __builtin_copysignf(q2, x);
}

// E4M3fn codes of four binary32 quotients (|r| < 464), round to nearest even, packed low to high.
__device__ __forceinline__ uint32_t e4m3fn_x4(float r0, float r1, float r2, float r3) {
    const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(r0, r1, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(r2, r3, lo, true);
}

// Maximum of v over each row of 16 lanes by DPP lane swaps (quad swaps, then the half-row and row
// mirrors): no LDS round trip.  Every lane of the row must be active.
__device__ __forceinline__ uint32_t row16_max(uint32_t v) {
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));   // quad_perm [1,0,3,2]
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));   // quad_perm [2,3,0,1]
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, false));  // row_half_mirror
    return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, false));  // row_mirror
}

// Maximum of v over the wave: its rows of 16 lanes, then the four row maxima by readlane.  Every lane
// must be active.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    v = row16_max(v);
    const uint32_t a = (uint32_t)__builtin_amdgcn_readlane((int)v, 0), b = (uint32_t)__builtin_amdgcn_readlane((int)v, 16);
    const uint32_t c = (uint32_t)__builtin_amdgcn_readlane((int)v, 32), d = (uint32_t)__builtin_amdgcn_readlane((int)v, 48);
    return max(max(a, b), max(c, d));
}

// scale of a block from its largest magnitude bit pattern
__device__ __forceinline__ float block_scale(uint32_t mag_max) {
    if (mag_max >= 0x7f800000u) return __uint_as_float(0x7fc00000u);
    const float s = __uint_as_float(mag_max) / 448.0f;
    return s == 0.0f ? 1.0f : s;
}
__device__ __forceinline__ float clamped_quotient(float x, float s) {
    return __builtin_amdgcn_fmed3f(x / s, -448.0f, 448.0f);
}

// One block of 128 BF16 values held by 16 lanes, eight each: this lane's eight codes, and the block's scale.
__device__ __forceinline__ uint2 quant_block_bf16x8(uint4 r, float& sc) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
    uint32_t mag = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) mag = max(mag, max((w[i] << 16) & 0x7fffffffu, w[i] & 0x7fff0000u));
    mag = row16_max(mag);
    sc = block_scale(mag);
    if (mag >= 0x7f800000u) return make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
    if (sc >= 0x1p-90f) {
        const float rc = 1.0f / sc;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = div_corrected(v[i], sc, rc);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = clamped_quotient(v[i], sc);
    }
    return make_uint2(e4m3fn_x4(v[0], v[1], v[2], v[3]), e4m3fn_x4(v[4], v[5], v[6], v[7]));
}

}  // namespace mx
