// 16-bit types and activations of the serving kernels.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace cqk {

template <bool F16>
__device__ __forceinline__ float to_f32(uint16_t b) {
    if constexpr (F16) return (float)__builtin_bit_cast(_Float16, b);
    return __uint_as_float((uint32_t)b << 16);
}

// Round to nearest even, NaN kept a NaN.
template <bool F16>
__device__ __forceinline__ uint16_t from_f32(float x) {
    if constexpr (F16) return __builtin_bit_cast(uint16_t, (_Float16)x);
    return __builtin_bit_cast(uint16_t, (__bf16)x);
}

enum { ACT_NONE = 0, ACT_RELU = 1, ACT_SILU = 2, ACT_GELU = 3, ACT_GELU_TANH = 4 };

// z / (1 + exp(-z)): the sigmoid of large negative z is exp(z), which keeps its relative accuracy
// until it underflows.
__device__ __forceinline__ float sigmoid(float z) { return 1.0f / (1.0f + __expf(-z)); }

// z N(z), N the normal distribution function: |z| (1 - N(|z|)) is subtracted from z, or is the negative of the value
// where z < 0 (z (1 + erf(z / sqrt 2)) / 2 cancels there: at -5 a tenth of it is gone, below -5.6 all).  The tail is
// 1 - N(a) = e^(-a^2 / 2) t p(t), t = 1 / (1 + 0.3 a): what is left of it without the exponential, over t, is smooth in t
// down to t -> 0, and p is its polynomial of degree 7 by reweighted least squares for a up to 14.5 (relative error
// 1.7e-7; behind it the exponential is 0).  8192 rows, 1024 -> 4096 with f32 outputs: 106 us, with erfcf
// 126, with 1 + erff 113.
__device__ __forceinline__ float gelu(float z) {
    const float a = fminf(fabsf(z), 20.0f);  // (an infinity times t would be a NaN)
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(a, 0.3f, 1.0f));
    float p = 0.0354238881f;
    p = __builtin_fmaf(p, t, -0.156159045f);
    p = __builtin_fmaf(p, t, 0.204557739f);
    p = __builtin_fmaf(p, t, -0.0520348236f);
    p = __builtin_fmaf(p, t, 0.12769216f);
    p = __builtin_fmaf(p, t, 0.100175842f);
    p = __builtin_fmaf(p, t, 0.120712151f);
    p = __builtin_fmaf(p, t, 0.119632006f);
    const float tail = a * t * (p * __builtin_amdgcn_exp2f(z * z * -0.72134752f));
    return z < 0.0f ? -tail : z - tail;  // (a NaN stays one)
}

template <int ACT>
__device__ __forceinline__ float activate(float z) {
    if constexpr (ACT == ACT_RELU) return z > 0.0f ? z : (z != z ? z : 0.0f);
    if constexpr (ACT == ACT_SILU) return z * sigmoid(z);
    if constexpr (ACT == ACT_GELU) return gelu(z);
    if constexpr (ACT == ACT_GELU_TANH) return z * sigmoid(1.5957691f * (z + 0.044715f * z * z * z));
    return z;
}

__device__ __forceinline__ float activate(int act, float z) {
    switch (act) {
        case ACT_RELU: return activate<ACT_RELU>(z);
        case ACT_SILU: return activate<ACT_SILU>(z);
        case ACT_GELU: return activate<ACT_GELU>(z);
        case ACT_GELU_TANH: return activate<ACT_GELU_TANH>(z);
        default: return z;
    }
}

// 16 bytes per lane from memory straight into LDS: lane l's to lds + 16 l (lds the same in all lanes).
// Written out, because the compiler's own form of it waits for every such load before the next read
// of LDS, also where that reads another buffer.  The caller waits (loaded_to_lds) before the barrier
// behind which the data is read.
__device__ __forceinline__ void load_to_lds(const void* from, const void* lds) {
    const uint32_t at = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)lds);
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(at), "v"(from) : "memory", "m0");
}
// The same from `base` (the same in all lanes) and a lane's own offset in bytes, below 2^32.
__device__ __forceinline__ void load_to_lds(const void* base, uint32_t offset, const void* lds) {
    const uint32_t at = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)lds);
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(at), "v"(offset), "s"(base) : "memory", "m0");
}
// The same with 4 bytes per lane.
__device__ __forceinline__ void load_to_lds_4(const void* from, const void* lds) {
    const uint32_t at = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)lds);
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(at), "v"(from) : "memory", "m0");
}
// Waits until at most LATER of the wave's loads are outstanding (they arrive in order).
template <int LATER = 0>
__device__ __forceinline__ void loaded_to_lds() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(LATER) : "memory");
}
// The same, and until the wave's reads of LDS are done; then a barrier of the workgroup's waves.  Reads of LDS in front of it
// see nothing of what is asked for behind it, those behind it all that the waves have waited for.
template <int LATER>
__device__ __forceinline__ void loaded_and_read() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(LATER) : "memory");
}

}  // namespace cqk
