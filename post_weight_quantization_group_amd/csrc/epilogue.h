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

}  // namespace cqk
