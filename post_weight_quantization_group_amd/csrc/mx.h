// Microscaled formats: blocks of 32 values with a shared power of two as a byte (e8m0, bias 127; 255: NaN) and elements
// of 4 bits (MXFP4, e2m1: 0 0.5 1 1.5 2 3 4 6, two a byte, the first in the low four bits) or 8 (MXFP8, e4m3: up to 448).
//
// gfx950 converts two elements an instruction from and to 16- and 32-bit values, with the scale as an fp32 operand of
// which it takes the exponent field (0: 2^-127, 255: NaN).  Checked over all codes, scales and bf16 and f16 values:
// decoding rounds once, to nearest even; encoding does too, and saturates for e2m1, but for e4m3 gives NaN above 464,
// so what exceeds 448 is cut to it before.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "serve_math.h"

namespace cqk {

enum { CACHE_16 = 0, MXFP4 = 3, MXFP8 = 4 };  // (as cq.h's types)
constexpr int MX_BLOCK = 32;

typedef __bf16 mx_bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 mx_f16x2 __attribute__((ext_vector_type(2)));
typedef short mx_s16x2 __attribute__((ext_vector_type(2)));
typedef float mx_f32x2 __attribute__((ext_vector_type(2)));
typedef uint16_t mx_u16x2 __attribute__((ext_vector_type(2)));

// floor(log2 of the largest element).
template <int FORM>
constexpr uint32_t mx_top_exponent() { return FORM == MXFP4 ? 2 : 8; }

// The scale byte of a block from the bits of its largest magnitude as fp32: 2^(floor(log2 top) - m), at least 2^-127;
// NaN where one of the values is an infinity or a NaN.
template <int FORM>
__device__ __forceinline__ uint32_t mx_scale_of(uint32_t top) {
    const uint32_t e = top >> 23;
    return e == 255 ? 255u : e > mx_top_exponent<FORM>() ? e - mx_top_exponent<FORM>() : 0u;
}
// The scale operand of the conversions.
__device__ __forceinline__ float mx_scale_operand(uint32_t byte) { return __uint_as_float(byte << 23); }

// ---- 16-bit values, four words of two
// The largest of a lane's eight magnitudes (as integers, which order them; infinities and NaNs on top).
__device__ __forceinline__ uint32_t mx_largest16(uint4 v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    mx_u16x2 most = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) most = __builtin_elementwise_max(most, __builtin_bit_cast(mx_u16x2, w[i] & 0x7fff7fffu));
    return most.x > most.y ? most.x : most.y;
}
// The larger of lanes' values over groups of four neighbouring lanes.
__device__ __forceinline__ uint32_t mx_most_of_four(uint32_t x) {
    uint32_t y = __builtin_amdgcn_update_dpp(0, x, 0xB1, 0xf, 0xf, false);  // lane XOR 1
    x = x > y ? x : y;
    y = __builtin_amdgcn_update_dpp(0, x, 0x4E, 0xf, 0xf, false);  // lane XOR 2
    return x > y ? x : y;
}
// A 16-bit magnitude as the bits of an fp32 value of the same value.
template <bool F16>
__device__ __forceinline__ uint32_t mx_as_f32(uint32_t magnitude) {
    if constexpr (F16) {
        const uint32_t b = __float_as_uint((float)__builtin_bit_cast(_Float16, (uint16_t)magnitude));
        return b;  // (infinity and NaN keep the exponent field of ones)
    }
    return magnitude << 16;
}
// Eight values of a block whose scale byte is `byte` as codes: one word (MXFP4) or two (MXFP8); 0 in a block of NaN.
template <int FORM, bool F16>
__device__ __forceinline__ uint2 mx_encode16(uint4 v, uint32_t byte) {
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
    // (for the lowest scale a subnormal operand: its exponent field is 0 as well, and it is the one checked)
    const float s = __uint_as_float(byte == 0 ? 0x00400000u : byte << 23);
    uint2 c = make_uint2(0, 0);
    if constexpr (FORM == MXFP4) {
        if constexpr (F16) {
            c.x = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c.x, __builtin_bit_cast(mx_f16x2, w[0]), s, 0);
            c.x = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c.x, __builtin_bit_cast(mx_f16x2, w[1]), s, 1);
            c.x = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c.x, __builtin_bit_cast(mx_f16x2, w[2]), s, 2);
            c.x = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c.x, __builtin_bit_cast(mx_f16x2, w[3]), s, 3);
        } else {
            c.x = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c.x, __builtin_bit_cast(mx_bf16x2, w[0]), s, 0);
            c.x = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c.x, __builtin_bit_cast(mx_bf16x2, w[1]), s, 1);
            c.x = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c.x, __builtin_bit_cast(mx_bf16x2, w[2]), s, 2);
            c.x = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c.x, __builtin_bit_cast(mx_bf16x2, w[3]), s, 3);
        }
    } else {
        // 448 scales, 1.75 2^8 2^(byte - 127), in the 16-bit type (where f16 cannot hold it, no value lies above it)
        const uint32_t limit32 = ((byte + 8) << 23) | 0x600000u;
        uint32_t limit = limit32 >> 16;
        if constexpr (F16) limit = __builtin_bit_cast(uint16_t, (_Float16)__uint_as_float(limit32));
        limit |= limit << 16;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = __builtin_bit_cast(uint32_t, __builtin_elementwise_min(__builtin_bit_cast(mx_u16x2, w[i] & 0x7fff7fffu),
                                                                         __builtin_bit_cast(mx_u16x2, limit))) |
                   (w[i] & 0x80008000u);
        mx_s16x2 lo = {0, 0}, hi = {0, 0};
        if constexpr (F16) {
            lo = __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(lo, __builtin_bit_cast(mx_f16x2, w[0]), s, false);
            lo = __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(lo, __builtin_bit_cast(mx_f16x2, w[1]), s, true);
            hi = __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(hi, __builtin_bit_cast(mx_f16x2, w[2]), s, false);
            hi = __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(hi, __builtin_bit_cast(mx_f16x2, w[3]), s, true);
        } else {
            lo = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(lo, __builtin_bit_cast(mx_bf16x2, w[0]), s, false);
            lo = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(lo, __builtin_bit_cast(mx_bf16x2, w[1]), s, true);
            hi = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(hi, __builtin_bit_cast(mx_bf16x2, w[2]), s, false);
            hi = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(hi, __builtin_bit_cast(mx_bf16x2, w[3]), s, true);
        }
        c = make_uint2(__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi));
    }
    if (byte == 255) c = make_uint2(0, 0);
    return c;
}

// ---- fp32 values
__device__ __forceinline__ uint32_t mx_largest32(const float* v) {
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t b = __float_as_uint(v[i]) & 0x7fffffffu;
        most = most > b ? most : b;
    }
    return most;
}
template <int FORM>
__device__ __forceinline__ uint2 mx_encode32(const float* v, uint32_t byte) {
    const float s = __uint_as_float(byte == 0 ? 0x00400000u : byte << 23);
    uint2 c = make_uint2(0, 0);
    if constexpr (FORM == MXFP4) {
        c.x = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c.x, v[0], v[1], s, 0);
        c.x = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c.x, v[2], v[3], s, 1);
        c.x = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c.x, v[4], v[5], s, 2);
        c.x = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c.x, v[6], v[7], s, 3);
    } else {
        const float limit = __uint_as_float(((byte + 8) << 23) | 0x600000u);
        float w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = fminf(fmaxf(v[i], -limit), limit);
        mx_s16x2 lo = {0, 0}, hi = {0, 0};
        lo = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(lo, w[0], w[1], s, false);
        lo = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(lo, w[2], w[3], s, true);
        hi = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(hi, w[4], w[5], s, false);
        hi = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(hi, w[6], w[7], s, true);
        c = make_uint2(__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi));
    }
    if (byte == 255) c = make_uint2(0, 0);
    return c;
}

// ---- back
// Eight values from a word of MXFP4 codes (of two words, MXFP8), times the scale, in the 16-bit type.
template <int FORM, bool F16>
__device__ __forceinline__ uint4 mx_decode16(uint2 c, float s) {
    uint32_t w[4];
    if constexpr (FORM == MXFP4) {
        if constexpr (F16) {
            w[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c.x, s, 0));
            w[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c.x, s, 1));
            w[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c.x, s, 2));
            w[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c.x, s, 3));
        } else {
            w[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c.x, s, 0));
            w[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c.x, s, 1));
            w[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c.x, s, 2));
            w[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c.x, s, 3));
        }
    } else {
        if constexpr (F16) {
            w[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c.x, s, false));
            w[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c.x, s, true));
            w[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c.y, s, false));
            w[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c.y, s, true));
        } else {
            w[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c.x, s, false));
            w[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c.x, s, true));
            w[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c.y, s, false));
            w[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c.y, s, true));
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
template <int FORM>
__device__ __forceinline__ void mx_decode32(uint2 c, float s, float* v) {
    mx_f32x2 p[4];
    if constexpr (FORM == MXFP4) {
        p[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c.x, s, 0);
        p[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c.x, s, 1);
        p[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c.x, s, 2);
        p[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c.x, s, 3);
    } else {
        p[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c.x, s, false);
        p[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c.x, s, true);
        p[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c.y, s, false);
        p[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c.y, s, true);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) v[2 * i] = p[i].x, v[2 * i + 1] = p[i].y;
}

}  // namespace cqk
