// Quantisation to microscaled blocks and back, of rows and of what goes into a paged cache, for gfx950.
//
// A block's scale and codes depend on its 32 values alone and hold no sums: nothing is rounded but the elements.  A
// lane takes 8 neighbouring values (16 bytes of 16-bit ones); the largest magnitude of a block comes from four
// neighbouring lanes by two data-parallel moves, and the conversions are the hardware's, two elements an instruction.
//
// Bound by memory.  8192 rows of 4096 bf16 values to MXFP4 14.4 us (84 MB with the codes: 5.8 TB/s, part of them from the
// caches; a copy of 1 GiB reaches 5.1 to 5.5), to MXFP8 17; f16 there and back, 8192 x 3584 by MXFP8, 15.0 us each way
// (89 MB, 5.9 TB/s).  Rows with gaps between them take as long (8192 x 4096 of rows of 3 x 4096 to MXFP4 12.9 us, to MXFP8 15.9,
// back into such rows 14.0 and 16.2; without gaps 14.3, 16.2, 13.7 and 16.2).  Few rows take a launch: 2.3 us, 3.8 there and back in a graph.
#include "mx.h"
#include "serve_args.h"

namespace cqk {
namespace {

template <int FORM>
__device__ __forceinline__ void store_codes(uint8_t* to, uint2 c) {
    if constexpr (FORM == MXFP4) *reinterpret_cast<uint32_t*>(to) = c.x;
    else *reinterpret_cast<uint2*>(to) = c;
}
template <int FORM>
__device__ __forceinline__ uint2 load_codes(const uint8_t* from) {
    if constexpr (FORM == MXFP4) return make_uint2(*reinterpret_cast<const uint32_t*>(from), 0);
    else return *reinterpret_cast<const uint2*>(from);
}
template <int FORM>
constexpr int code_bytes() { return FORM == MXFP4 ? 4 : 8; }  // of eight values

// Rows [rows][len]: a thread per 8 values.  FLAT: the rows follow each other without gaps, in every array.
template <int FORM, int TYPE, bool FLAT>
__global__ __launch_bounds__(256) void quantize_kernel(MxRowsArgs a) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, per_row = a.len / 8;
    if (i >= per_row * a.rows) return;
    const int64_t row = FLAT ? 0 : i / per_row, at = FLAT ? i : i % per_row;
    uint32_t byte;
    uint2 c;
    if constexpr (TYPE == 2) {
        const float4* from = reinterpret_cast<const float4*>(static_cast<const float*>(a.values) + row * a.ldx + 8 * at);
        const float4 lo = from[0], hi = from[1];
        const float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        byte = mx_scale_of<FORM>(mx_most_of_four(mx_largest32(v)));
        c = mx_encode32<FORM>(v, byte);
    } else {
        const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.values) + row * a.ldx + 8 * at);
        byte = mx_scale_of<FORM>(mx_as_f32<TYPE == 1>(mx_most_of_four(mx_largest16(v))));
        c = mx_encode16<FORM, TYPE == 1>(v, byte);
    }
    store_codes<FORM>(a.codes + row * a.ldc + at * code_bytes<FORM>(), c);
    if (at % 4 == 0) a.scales[row * a.lds + at / 4] = (uint8_t)byte;
}

template <int FORM, int TYPE, bool FLAT>
__global__ __launch_bounds__(256) void dequantize_kernel(MxRowsArgs a) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, per_row = a.len / 8;
    if (i >= per_row * a.rows) return;
    const int64_t row = FLAT ? 0 : i / per_row, at = FLAT ? i : i % per_row;
    const uint2 c = load_codes<FORM>(a.codes + row * a.ldc + at * code_bytes<FORM>());
    const float s = mx_scale_operand(a.scales[row * a.lds + at / 4]);
    if constexpr (TYPE == 2) {
        float v[8];
        mx_decode32<FORM>(c, s, v);
        float4* to = reinterpret_cast<float4*>(static_cast<float*>(a.values) + row * a.ldx + 8 * at);
        to[0] = make_float4(v[0], v[1], v[2], v[3]);
        to[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.values) + row * a.ldx + 8 * at) = mx_decode16<FORM, TYPE == 1>(c, s);
    }
}

// New keys and values into the pages: 8 values of a key and of a value a thread, which finds their slot itself.  16,384
// tokens of 8 heads of 128: 16.7 us to MXFP4 (85 MB, 5.1 TB/s); 64 tokens 2.6 us in a graph, a launch.  WIDE: they move 16
// bytes at a time.
template <bool WIDE>
__device__ __forceinline__ uint4 eight(const uint16_t* p) {
    if constexpr (WIDE) return *reinterpret_cast<const uint4*>(p);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = p[2 * i] | (uint32_t)p[2 * i + 1] << 16;
    return make_uint4(w[0], w[1], w[2], w[3]);
}
template <int FORM, bool F16, bool WIDE>
__global__ __launch_bounds__(256) void cache_write_mx_kernel(MxCacheWriteArgs a) {
    const uint32_t per_row = a.c.D / 8, i = blockIdx.x * 256 + threadIdx.x;  // (below 2^31 + 256)
    const uint32_t row = i / per_row, piece = i % per_row, t = row / a.c.H, h = row % a.c.H;
    if (t >= (uint32_t)a.T) return;
    const int32_t slot = a.slots[t];
    if (slot < 0 || slot >= a.n_slots) return;
    const uint4 k = eight<WIDE>(a.k + t * a.k_tok + h * a.k_head + 8 * piece);
    const uint4 v = eight<WIDE>(a.v + t * a.v_tok + h * a.v_head + 8 * piece);
    const uint32_t page = (uint32_t)slot / (uint32_t)a.c.page, at = (uint32_t)slot % (uint32_t)a.c.page;
    const int64_t to = page * a.c.c_page + h * a.c.c_head + at * a.c.c_row + piece * code_bytes<FORM>();
    const int64_t scale = page * a.c.s_page + h * a.c.s_head + at * a.c.s_row + piece / 4;
    const uint32_t kb = mx_scale_of<FORM>(mx_as_f32<F16>(mx_most_of_four(mx_largest16(k))));
    const uint32_t vb = mx_scale_of<FORM>(mx_as_f32<F16>(mx_most_of_four(mx_largest16(v))));
    store_codes<FORM>(a.c.kc + to, mx_encode16<FORM, F16>(k, kb));
    store_codes<FORM>(a.c.vc + to, mx_encode16<FORM, F16>(v, vb));
    if (piece % 4 == 0) {
        a.c.ks[scale] = (uint8_t)kb;
        a.c.vs[scale] = (uint8_t)vb;
    }
}

template <int FORM, int TYPE>
hipError_t rows_of_type(const MxRowsArgs& a, bool back, hipStream_t st) {
    const bool flat = a.rows == 1;
    const int64_t blocks = (a.rows * (a.len / 8) + 255) / 256;
    const dim3 grid((unsigned)blocks);
    if (back && flat) hipLaunchKernelGGL((dequantize_kernel<FORM, TYPE, true>), grid, dim3(256), 0, st, a);
    else if (back) hipLaunchKernelGGL((dequantize_kernel<FORM, TYPE, false>), grid, dim3(256), 0, st, a);
    else if (flat) hipLaunchKernelGGL((quantize_kernel<FORM, TYPE, true>), grid, dim3(256), 0, st, a);
    else hipLaunchKernelGGL((quantize_kernel<FORM, TYPE, false>), grid, dim3(256), 0, st, a);
    return hipGetLastError();
}

template <int FORM>
hipError_t rows_of_form(const MxRowsArgs& a, bool back, hipStream_t st) {
    switch (a.type) {
        case 0: return rows_of_type<FORM, 0>(a, back, st);
        case 1: return rows_of_type<FORM, 1>(a, back, st);
        default: return rows_of_type<FORM, 2>(a, back, st);
    }
}

template <int FORM>
hipError_t write_of_form(const MxCacheWriteArgs& a, hipStream_t st) {
    const int64_t strides = a.k_tok | a.k_head | a.v_tok | a.v_head;
    const bool wide = strides % 8 == 0 && ((uintptr_t)a.k | (uintptr_t)a.v) % 16 == 0;
    const dim3 grid((unsigned)(((int64_t)a.T * a.c.H * (a.c.D / 8) + 255) / 256));
    if (a.f16 && wide) hipLaunchKernelGGL((cache_write_mx_kernel<FORM, true, true>), grid, dim3(256), 0, st, a);
    else if (a.f16) hipLaunchKernelGGL((cache_write_mx_kernel<FORM, true, false>), grid, dim3(256), 0, st, a);
    else if (wide) hipLaunchKernelGGL((cache_write_mx_kernel<FORM, false, true>), grid, dim3(256), 0, st, a);
    else hipLaunchKernelGGL((cache_write_mx_kernel<FORM, false, false>), grid, dim3(256), 0, st, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_rows(const MxRowsArgs& args, bool back, hipStream_t st) {
    MxRowsArgs a = args;
    if (a.ldx == a.len && a.ldc == a.len / (a.form == MXFP4 ? 2 : 1) && a.lds == a.len / MX_BLOCK) {
        a.len *= a.rows;
        a.rows = 1;
    }
    return a.form == MXFP4 ? rows_of_form<MXFP4>(a, back, st) : rows_of_form<MXFP8>(a, back, st);
}

hipError_t launch_cache_write_mx(const MxCacheWriteArgs& a, hipStream_t st) {
    return a.c.form == MXFP4 ? write_of_form<MXFP4>(a, st) : write_of_form<MXFP8>(a, st);
}

}  // namespace cqk
