// Linear layer over GPTQ-v1 tensors with its epilogue, the simple form: a thread per output.
#include "serve_args.h"
#include "serve_math.h"

namespace cqk {
namespace {

template <bool F16>
__device__ float column(const LinearArgs& a, int64_t m, int64_t o, int64_t cols) {
    float z = 0.0f;
    for (int64_t g = 0; g < a.in / 128; ++g) {
        float part = 0.0f;
        for (int r = 0; r < 16; ++r) {
            const uint32_t w = (uint32_t)a.qw[(g * 16 + r) * cols + o];
            const uint16_t* xr = a.x + m * a.ldx + g * 128 + r * 8;
            for (int j = 0; j < 8; ++j)
                part = __builtin_fmaf(to_f32<F16>(xr[j]), (float)((int)((w >> (4 * j)) & 15) - 8), part);
        }
        z = __builtin_fmaf(to_f32<true>(a.scales[g * cols + o]), part, z);
    }
    if (a.bias) z += to_f32<F16>(a.bias[o]);
    return z;
}

template <bool F16>
__global__ __launch_bounds__(256) void linear_kernel(LinearArgs a) {
    const int64_t o = (int64_t)blockIdx.y * 64 + (threadIdx.x & 63), m = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (o >= a.out || m >= a.M) return;
    const int64_t cols = a.gated ? 2 * a.out : a.out;
    float z = activate(a.act, column<F16>(a, m, o, cols));
    if (a.gated) z *= column<F16>(a, m, o + a.out, cols);
    if (a.residual) z += to_f32<F16>(a.residual[m * a.ldr + o]);
    if (a.y_f32) ((float*)a.y)[m * a.ldy + o] = z;
    else ((uint16_t*)a.y)[m * a.ldy + o] = from_f32<F16>(z);
}

}  // namespace

hipError_t launch_linear(const LinearArgs& a, hipStream_t st) {
    const dim3 grid((unsigned)((a.M + 3) / 4), (unsigned)((a.out + 63) / 64));
    if (a.x_f16) hipLaunchKernelGGL(linear_kernel<true>, grid, dim3(256), 0, st, a);
    else hipLaunchKernelGGL(linear_kernel<false>, grid, dim3(256), 0, st, a);
    return hipGetLastError();
}

}  // namespace cqk
