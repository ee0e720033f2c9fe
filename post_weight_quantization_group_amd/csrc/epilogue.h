// The linear layers' epilogue: bias, activation, gate, residual and the rounding into the output's type, in fp32.
// Args holds bias, residual (of the 16-bit type), y, ldr, ldy, M, out, act, gated and y_f32, as LinearArgs.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "serve_math.h"

namespace cqk {

typedef float f32x4 __attribute__((ext_vector_type(4)));

// act(z + b) [* (z' + b')] + r of output (m, o) and its store.
template <bool F16, typename Args>
__device__ __forceinline__ void finish(const Args& a, int64_t m, int64_t o, float z, float up) {
    if (a.bias) z += to_f32<F16>(a.bias[o]);
    z = activate(a.act, z);
    if (a.gated) {
        if (a.bias) up += to_f32<F16>(a.bias[a.out + o]);
        z *= up;
    }
    if (a.residual) z += to_f32<F16>(a.residual[m * a.ldr + o]);
    if (a.y_f32) reinterpret_cast<float*>(a.y)[m * a.ldy + o] = z;
    else reinterpret_cast<uint16_t*>(a.y)[m * a.ldy + o] = from_f32<F16>(z);
}

// Whether four neighbouring outputs from a multiple of 4 on can be moved at once.
template <typename Args>
__device__ __forceinline__ bool outputs_in_fours(const Args& a) {
    bool ok = a.out % 4 == 0 && a.ldy % 4 == 0 && ((uintptr_t)a.y & (a.y_f32 ? 15 : 7)) == 0;
    if (a.residual) ok = ok && a.ldr % 4 == 0 && ((uintptr_t)a.residual & 7) == 0;
    if (a.bias) ok = ok && ((uintptr_t)a.bias & 7) == 0;
    return ok;
}

template <bool F16>
__device__ __forceinline__ f32x4 four(const uint16_t* p) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    return f32x4{to_f32<F16>((uint16_t)v.x), to_f32<F16>((uint16_t)(v.x >> 16)), to_f32<F16>((uint16_t)v.y),
                 to_f32<F16>((uint16_t)(v.y >> 16))};
}

// finish() of the outputs (m, o .. o + 3) that exist.
template <bool F16, typename Args>
__device__ __forceinline__ void finish4(const Args& a, int64_t m, int64_t o, f32x4 z, f32x4 up, bool wide) {
    if (m >= a.M || o >= a.out) return;
    if (!wide) {
        for (int e = 0; e < 4; ++e)
            if (o + e < a.out) finish<F16>(a, m, o + e, z[0], up[0]), z = z.yzwx, up = up.yzwx;
        return;
    }
    if (a.bias) {
        z += four<F16>(a.bias + o);
        if (a.gated) up += four<F16>(a.bias + a.out + o);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) z[e] = activate(a.act, z[e]);
    if (a.gated) z *= up;
    if (a.residual) z += four<F16>(a.residual + m * a.ldr + o);
    if (a.y_f32) {
        *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(a.y) + m * a.ldy + o) = z;
    } else {
        uint32_t b[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) b[e] = from_f32<F16>(z[e]);
        *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.y) + m * a.ldy + o) =
            make_uint2(b[0] | b[1] << 16, b[2] | b[3] << 16);
    }
}

// Whether eight neighbouring outputs from a multiple of 8 on can be moved at once.
template <typename Args>
__device__ __forceinline__ bool outputs_in_eights(const Args& a) {
    bool ok = a.out % 8 == 0 && a.ldy % 8 == 0 && ((uintptr_t)a.y & 15) == 0;
    if (a.residual) ok = ok && a.ldr % 8 == 0 && ((uintptr_t)a.residual & 15) == 0;
    if (a.bias) ok = ok && ((uintptr_t)a.bias & 15) == 0;
    return ok;
}

template <bool F16>
__device__ __forceinline__ void eight(uint4 v, float* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[2 * i] = to_f32<F16>((uint16_t)w[i]), f[2 * i + 1] = to_f32<F16>((uint16_t)(w[i] >> 16));
}

__device__ __forceinline__ void activate8(int act, float* z) {
    switch (act) {
        case ACT_RELU:
#pragma unroll
            for (int e = 0; e < 8; ++e) z[e] = activate<ACT_RELU>(z[e]);
            break;
        case ACT_SILU:
#pragma unroll
            for (int e = 0; e < 8; ++e) z[e] = activate<ACT_SILU>(z[e]);
            break;
        case ACT_GELU:
#pragma unroll
            for (int e = 0; e < 8; ++e) z[e] = activate<ACT_GELU>(z[e]);
            break;
        case ACT_GELU_TANH:
#pragma unroll
            for (int e = 0; e < 8; ++e) z[e] = activate<ACT_GELU_TANH>(z[e]);
            break;
        default: break;
    }
}

// finish() of ROWS rows of eight neighbouring outputs each, from column o on, z and (gated) up in LDS; the rows are
// `row_of(i)`, their sums at `from(i)`, those of the other half UP floats further on.  All residuals are asked for before the
// first is used: `residuals` holds them, from Residuals::ask.
template <int ROWS>
struct Residuals {
    uint4 v[ROWS];
    template <typename Args, typename Row>
    __device__ __forceinline__ void ask(const Args& a, int64_t o, Row row_of) {
        if (!a.residual) return;
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const int64_t m = row_of(i);
            v[i] = *reinterpret_cast<const uint4*>(a.residual + (m < a.M ? m : a.M - 1) * a.ldr + o);
        }
    }
};
template <bool F16, int UP, int ROWS, typename Args, typename Row, typename From>
__device__ __forceinline__ void finish8(const Args& a, int64_t o, const float* bias, const float* up_bias,
                                        const Residuals<ROWS>& residuals, Row row_of, From from) {
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int64_t m = row_of(i);
        const __attribute__((address_space(3))) float* at = from(i);
        float z[8], up[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] = at[e] + bias[e];
        activate8(a.act, z);
        if (a.gated) {
#pragma unroll
            for (int e = 0; e < 8; ++e) up[e] = at[UP + e] + up_bias[e];
#pragma unroll
            for (int e = 0; e < 8; ++e) z[e] *= up[e];
        }
        if (a.residual) {
            float r[8];
            eight<F16>(residuals.v[i], r);
#pragma unroll
            for (int e = 0; e < 8; ++e) z[e] += r[e];
        }
        if (m >= a.M) continue;
        if (a.y_f32) {
            f32x4* to = reinterpret_cast<f32x4*>(reinterpret_cast<float*>(a.y) + m * a.ldy + o);
            to[0] = f32x4{z[0], z[1], z[2], z[3]};
            to[1] = f32x4{z[4], z[5], z[6], z[7]};
        } else {
            uint32_t b[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) b[e] = from_f32<F16>(z[e]);
            *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.y) + m * a.ldy + o) =
                make_uint4(b[0] | b[1] << 16, b[2] | b[3] << 16, b[4] | b[5] << 16, b[6] | b[7] << 16);
        }
    }
}

}  // namespace cqk
