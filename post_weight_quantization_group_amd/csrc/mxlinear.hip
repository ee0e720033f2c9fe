// Linear layer over MXFP4 weights with its epilogue, for gfx950:
//
//   z[m][c] = sum_k Q(x)[m][k] W[c][k],    y = act(z + b) [* (z' + b')] + r,
//
// Q(x) being x's rows in MXFP4 or MXFP8.  The products run on the matrix cores in those formats as they are stored,
// two blocks of 32 (or four) an instruction with their scales as operands: exact products, fp32 sums.
//
// Lane layouts (checked on gfx950), A and B alike; D as of the 16-bit instructions.  16x16x128: lane l holds row l % 16;
// of 4-bit elements k = 32 (l / 16) .. + 31, of 8-bit ones 16 (l / 16) .. + 15 and 64 + 16 (l / 16) .. + 15; and in
// either case the scale of k = 32 (l / 16) .. + 31.  32x32x64: row l % 32, 4-bit k = 32 (l / 32) .. + 31, 8-bit
// 16 (l / 32) .. + 15 and 32 + 16 (l / 32) .. + 15, the scale that of k = 32 (l / 32) .. + 31.
// W is the A operand: a lane then has neighbouring outputs of one row.
//
// Sums of 4-bit products are fp32 throughout (within 2^-23 of the sum of magnitudes, an instruction).  With 8-bit
// elements the products of a lane's 16 neighbouring ones are aligned to the largest of them and cut some 15 bits below its
// leading one: 2688 and -2688 beside 0.06 leave 0, and sums are off by up to 2^-13 of the sum of magnitudes.  So an e4m3
// operand goes in twice: its elements of 2 and more (bit 6 of their codes), whose products with e2m1 ones span
// the 15 bits from 2^11 to 2^-3, and the others, from 2^3 to 2^-10.  Both sums are then exact in a lane, and fp32 beyond.
#include "epilogue.h"
#include "mx.h"
#include "serve_args.h"

namespace cqk {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ i32x8 operand(uint4 lo, uint4 hi = make_uint4(0, 0, 0, 0)) {
    return i32x8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
}

// The e4m3 elements of 2 and more in magnitude; the others are what is left.
__device__ __forceinline__ i32x8 large_elements(i32x8 v) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t large = (uint32_t)v[i] & 0x40404040u;
        v[i] &= (int)((large << 2) - (large >> 6));  // 0xff in their bytes
    }
    return v;
}
// acc += W x, 16 by 16 over 128 of k.
template <int FORM>
__device__ __forceinline__ f32x4 add_products(i32x8 w, int ws, i32x8 x, int xs, f32x4 acc) {
    if constexpr (FORM == MXFP4)
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, acc, 4, 4, 0, ws, 0, xs);
    const i32x8 large = large_elements(x);
    acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x ^ large, acc, 4, 0, 0, ws, 0, xs);
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, large, acc, 4, 0, 0, ws, 0, xs);
}

// ---------------------------------------------------------------------------------------------
// Few rows, or few tiles: a workgroup takes 16 MT rows and 16 CT columns (gated: half of them of the gate, the others
// of the other half), its W waves every W-th 128 of k; their sums join in LDS in the order of the waves.  Weights and
// x go straight into the lanes that multiply them.  x of 16 bits is quantized there, each block by the lane, or
// the two lanes, that hold it.
enum { X_BF16 = 0, X_F16 = 1, X_CODES = 2 };

// A row tile's x operand of 128 k: what is loaded, and what the matrix cores take.
template <int FORM, int XT>
struct XPart {
    uint4 v[XT == X_CODES ? (FORM == MXFP4 ? 1 : 2) : 4];
    uint8_t byte;
    __device__ __forceinline__ void load(const MxLinearArgs& a, int64_t m, int step, int quad) {
        if constexpr (XT == X_CODES) {
            const uint8_t* x = static_cast<const uint8_t*>(a.x) + m * a.ldx;
            if constexpr (FORM == MXFP4) {
                v[0] = *reinterpret_cast<const uint4*>(x + (int64_t)step * 64 + 16 * quad);
            } else {
                v[0] = *reinterpret_cast<const uint4*>(x + (int64_t)step * 128 + 16 * quad);
                v[1] = *reinterpret_cast<const uint4*>(x + (int64_t)step * 128 + 64 + 16 * quad);
            }
            byte = a.xs[m * a.ldxs + 4 * step + quad];
        } else {
            const uint4* x = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.x) + m * a.ldx + (int64_t)step * 128);
            if constexpr (FORM == MXFP4) {  // the lane's own block
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = x[4 * quad + i];
            } else {  // half of block quad / 2 and half of block 2 + quad / 2
                v[0] = x[2 * quad];
                v[1] = x[2 * quad + 1];
                v[2] = x[8 + 2 * quad];
                v[3] = x[8 + 2 * quad + 1];
            }
        }
    }
    __device__ __forceinline__ i32x8 take(int quad, int& scale) const {
        constexpr bool F16 = XT == X_F16;
        if constexpr (XT == X_CODES) {
            scale = byte;
            if constexpr (FORM == MXFP4) return operand(v[0]);
            else return operand(v[0], v[1]);
        } else if constexpr (FORM == MXFP4) {
            uint32_t most = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t x = mx_largest16(v[i]);
                most = most > x ? most : x;
            }
            const uint32_t b = mx_scale_of<FORM>(mx_as_f32<F16>(most));
            scale = b;
            return operand(make_uint4(mx_encode16<FORM, F16>(v[0], b).x, mx_encode16<FORM, F16>(v[1], b).x,
                                      mx_encode16<FORM, F16>(v[2], b).x, mx_encode16<FORM, F16>(v[3], b).x));
        } else {
            uint32_t a = mx_largest16(v[0]), c = mx_largest16(v[1]), d = mx_largest16(v[2]), e = mx_largest16(v[3]);
            a = a > c ? a : c;
            d = d > e ? d : e;
            const uint32_t own = a | d << 16, other = __shfl_xor(own, 16);
            const mx_u16x2 most = __builtin_elementwise_max(__builtin_bit_cast(mx_u16x2, own), __builtin_bit_cast(mx_u16x2, other));
            const uint32_t b0 = mx_scale_of<FORM>(mx_as_f32<F16>(most.x)), b1 = mx_scale_of<FORM>(mx_as_f32<F16>(most.y));
            // lanes 16 .. 31 of the wave hold block 2's scale and need block 1's, lanes 32 .. 47 the other way round
            const uint32_t passed = __shfl_xor(quad < 2 ? b1 : b0, 48);
            scale = quad == 0 ? b0 : quad == 3 ? b1 : passed;
            const uint2 c0 = mx_encode16<FORM, F16>(v[0], b0), c1 = mx_encode16<FORM, F16>(v[1], b0);
            const uint2 c2 = mx_encode16<FORM, F16>(v[2], b1), c3 = mx_encode16<FORM, F16>(v[3], b1);
            return operand(make_uint4(c0.x, c0.y, c1.x, c1.y), make_uint4(c2.x, c2.y, c3.x, c3.y));
        }
    }
};

template <int FORM, int XT, bool F16, int MT, int CT, int W>
__global__ __launch_bounds__(64 * W) void few_rows_mx(MxLinearArgs a, int col_tiles) {
    __shared__ __align__(16) float sums[W * MT * 16 * CT * 16];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, col = lane & 15, quad = lane >> 4;
    const int64_t ct = blockIdx.x % col_tiles, rt = blockIdx.x / col_tiles;
    const int per = a.gated ? 8 * CT : 16 * CT;  // outputs per workgroup
    const int64_t n0 = ct * per, m0 = rt * (16 * MT);
    const uint8_t *wp[CT], *sp[CT];
#pragma unroll
    for (int t = 0; t < CT; ++t) {
        const bool up = a.gated && t >= CT / 2;
        const int64_t o = n0 + 16 * (up ? t - CT / 2 : t) + col;
        const int64_t c = (o < a.out ? o : a.out - 1) + (up ? a.out : 0);  // (past the edge: the last one)
        wp[t] = a.w + c * (a.in / 2) + 16 * quad;
        sp[t] = a.ws + c * (a.in / MX_BLOCK) + quad;
    }
    int64_t row[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int64_t m = m0 + 16 * i + col;
        row[i] = m < a.M ? m : a.M - 1;
    }
    const int steps = (int)(a.in / 128);
    uint4 w[CT];
    uint8_t ws[CT];
    XPart<FORM, XT> x[MT];
    auto fetch = [&](int s) {
        if (s >= steps) return;
#pragma unroll
        for (int t = 0; t < CT; ++t) {
            w[t] = *reinterpret_cast<const uint4*>(wp[t] + (int64_t)s * 64);
            ws[t] = sp[t][4 * s];
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) x[i].load(a, row[i], s, quad);
    };
    f32x4 acc[MT][CT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int t = 0; t < CT; ++t) acc[i][t] = f32x4{0, 0, 0, 0};
    fetch(wave);
    for (int s = wave; s < steps; s += W) {
        uint4 wn[CT];
        int wsn[CT];
        XPart<FORM, XT> xn[MT];
#pragma unroll
        for (int t = 0; t < CT; ++t) wn[t] = w[t], wsn[t] = ws[t];
#pragma unroll
        for (int i = 0; i < MT; ++i) xn[i] = x[i];
        fetch(s + W);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            int xs;
            const i32x8 b = xn[i].take(quad, xs);
#pragma unroll
            for (int t = 0; t < CT; ++t)
                acc[i][t] = add_products<FORM>(operand(wn[t]), wsn[t], b, xs, acc[i][t]);
        }
    }
    // sums[wave][row][16 t + column]
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int t = 0; t < CT; ++t)
            *reinterpret_cast<f32x4*>(&sums[((wave * MT + i) * 16 + col) * (16 * CT) + 16 * t + 4 * quad]) = acc[i][t];
    __syncthreads();
    for (int i = tid; i < MT * 16 * per; i += 64 * W) {
        const int r = i / per, n = i % per;
        const int64_t m = m0 + r, o = n0 + n;
        if (m >= a.M || o >= a.out) continue;
        float z = 0.0f, up = 0.0f;
#pragma unroll
        for (int v = 0; v < W; ++v) {
            z += sums[(v * MT * 16 + r) * (16 * CT) + n];
            if (a.gated) up += sums[(v * MT * 16 + r) * (16 * CT) + 8 * CT + n];
        }
        finish<F16>(a, m, o, z, up);
    }
}

template <int FORM, int XT, bool F16, int MT, int CT, int W>
hipError_t few(const MxLinearArgs& a, hipStream_t st) {
    const int per = a.gated ? 8 * CT : 16 * CT;
    const int64_t ct = (a.out + per - 1) / per, rt = (a.M + 16 * MT - 1) / (16 * MT);
    hipLaunchKernelGGL((few_rows_mx<FORM, XT, F16, MT, CT, W>), dim3((unsigned)(ct * rt)), dim3(64 * W), 0, st, a, (int)ct);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------------------------
// Many rows: a workgroup takes BIG_M rows of x's codes and BIG_N rows of W (gated: half of them of the gate, the others of the
// other half), 128 of k a step; its four waves 64 by 128 each, as 2 x 4 products of 32 x 32.  Codes and scales go from
// memory straight into LDS, some steps ahead, one barrier a step.  16-byte pieces of a row lie turned in it by the row's
// number, so that the rows which a quarter of a wave reads at once are in different banks.
constexpr int BIG_M = 128, BIG_N = 256;

template <int FORM>
__device__ __forceinline__ f32x16 add_products_32(i32x8 w, int ws, i32x8 x, i32x8 large, int xs, f32x16 acc, bool high) {
    if constexpr (FORM == MXFP4) {
        if (high) return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w, x, acc, 4, 4, 2, ws, 2, xs);
        return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w, x, acc, 4, 4, 0, ws, 0, xs);
    } else if (high) {
        acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w, x, acc, 4, 0, 2, ws, 2, xs);
        return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w, large, acc, 4, 0, 2, ws, 2, xs);
    } else {
        acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w, x, acc, 4, 0, 0, ws, 0, xs);
        return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w, large, acc, 4, 0, 0, ws, 0, xs);
    }
}

template <int FORM, bool F16>
__global__ __launch_bounds__(256, 2) void many_rows_mx(MxLinearArgs a, int row_tiles, int col_tiles) {
    constexpr int STAGES = FORM == MXFP4 ? 3 : 2;
    constexpr int X_ROW = FORM == MXFP4 ? 64 : 128;  // bytes of a step's row of x; 64 of W
    constexpr int X_LOADS = BIG_M * X_ROW / 1024 / 4, LOADS = 4 + X_LOADS + 2;  // a wave's a step
    constexpr int LINE = BIG_N + 4;                                            // floats of a row in the epilogue
    struct Stage {
        uint8_t w[BIG_N * 64], x[BIG_M * X_ROW];
        uint32_t ws[BIG_N], xs[2 * BIG_M];  // (the upper half: the same scales again, so that every wave loads as much)
    };
    constexpr int BYTES = STAGES * sizeof(Stage) > 64 * LINE * 4 ? STAGES * sizeof(Stage) : 64 * LINE * 4;
    __shared__ __align__(1024) uint8_t lds[BYTES];
    Stage* stage = reinterpret_cast<Stage*>(lds);
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 31, half = lane >> 5, wr = wave & 1, wc = wave >> 1;
    // Workgroups go to the eight XCDs in turn: each XCD takes a run of tiles, in bands of 8 row tiles, so that the tiles
    // it works on at a time share rows of x and W in its L2.
    int64_t id = blockIdx.x;
    {
        const int64_t all = (int64_t)row_tiles * col_tiles, base = all / 8, more = all % 8, x = id % 8, j = id / 8;
        id = x * base + (x < more ? x : more) + j;
    }
    const int64_t band = id / (8 * col_tiles), in_band = id % (8 * col_tiles);
    const int64_t high = row_tiles - band * 8 < 8 ? row_tiles - band * 8 : 8;
    const int64_t rt = band * 8 + in_band % high, ct = in_band / high;
    const int per = a.gated ? BIG_N / 2 : BIG_N;  // outputs per workgroup
    const int64_t m0 = rt * BIG_M, n0 = ct * per;
    // row of W for row i of the tile; past the edge the last one
    auto w_row = [&](int i) {
        const bool up = a.gated && i >= BIG_N / 2;
        const int64_t o = n0 + (up ? i - BIG_N / 2 : i);
        return (o < a.out ? o : a.out - 1) + (up ? a.out : 0);
    };
    auto x_row = [&](int i) { return m0 + i < a.M ? m0 + i : a.M - 1; };
    const int steps = (int)(a.in / 128);
    const uint8_t *wp[4], *xp[X_LOADS], *wsp, *xsp;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = 64 * wave + 16 * i + lane / 4;
        wp[i] = a.w + w_row(row) * (a.in / 2) + 16 * ((lane & 3) ^ ((row >> 2) & 3));
    }
#pragma unroll
    for (int i = 0; i < X_LOADS; ++i) {
        if constexpr (FORM == MXFP4) {
            const int row = 32 * wave + 16 * i + lane / 4;
            xp[i] = static_cast<const uint8_t*>(a.x) + x_row(row) * a.ldx + 16 * ((lane & 3) ^ ((row >> 2) & 3));
        } else {
            const int row = 32 * wave + 8 * i + lane / 8;
            xp[i] = static_cast<const uint8_t*>(a.x) + x_row(row) * a.ldx + 16 * ((lane & 7) ^ ((row >> 1) & 7));
        }
    }
    wsp = a.ws + w_row(64 * wave + lane) * (a.in / MX_BLOCK);
    xsp = a.xs + x_row(64 * (wave & 1) + lane) * a.ldxs;
    auto ask = [&](int s) {
        Stage& t = stage[s % STAGES];
#pragma unroll
        for (int i = 0; i < 4; ++i) load_to_lds(wp[i] + (int64_t)s * 64, &t.w[(64 * wave + 16 * i) * 64]);
#pragma unroll
        for (int i = 0; i < X_LOADS; ++i)
            load_to_lds(xp[i] + (int64_t)s * X_ROW, &t.x[(32 * wave + (FORM == MXFP4 ? 16 : 8) * i) * X_ROW]);
        load_to_lds_4(wsp + 4 * s, &t.ws[64 * wave]);
        load_to_lds_4(xsp + 4 * s, &t.xs[64 * wave]);
    };
    f32x16 acc[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
    for (int s = 0; s < STAGES - 1 && s < steps; ++s) ask(s);
    for (int s = 0; s < steps; ++s) {
        if (s + STAGES - 2 < steps) loaded_to_lds<(STAGES - 2) * LOADS>();
        else loaded_to_lds<0>();
        __syncthreads();  // this step's codes are in LDS, and the previous step's have been read
        if (s + STAGES - 1 < steps) ask(s + STAGES - 1);
        const Stage& t = stage[s % STAGES];
        int ws[4], xs[2];
#pragma unroll
        for (int i = 0; i < 4; ++i) ws[i] = (int)(t.ws[128 * wc + 32 * i + r] >> (8 * half));
#pragma unroll
        for (int j = 0; j < 2; ++j) xs[j] = (int)(t.xs[64 * wr + 32 * j + r] >> (8 * half));
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            i32x8 w[4], x[2], large[2];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = operand(*reinterpret_cast<const uint4*>(&t.w[(128 * wc + 32 * i + r) * 64 + 16 * ((2 * ks + half) ^ ((r >> 2) & 3))]));
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint8_t* row = &t.x[(64 * wr + 32 * j + r) * X_ROW];
                if constexpr (FORM == MXFP4) {
                    x[j] = operand(*reinterpret_cast<const uint4*>(row + 16 * ((2 * ks + half) ^ ((r >> 2) & 3))));
                    large[j] = x[j];
                } else {
                    x[j] = operand(*reinterpret_cast<const uint4*>(row + 16 * ((4 * ks + half) ^ ((r >> 1) & 7))),
                                   *reinterpret_cast<const uint4*>(row + 16 * ((4 * ks + 2 + half) ^ ((r >> 1) & 7))));
                    large[j] = large_elements(x[j]);
                    x[j] ^= large[j];
                }
            }
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[i][j] = add_products_32<FORM>(w[i], ws[i], x[j], large[j], xs[j], acc[i][j], ks);
        }
    }
    // The epilogue, 32 rows of every wave at a time through LDS: a thread then has four neighbouring outputs of a row, and
    // residual and y move in whole lines.
    const bool wide = outputs_in_fours(a);
    float* tile = reinterpret_cast<float*>(lds);  // [64][LINE]
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 16; e += 4)
                *reinterpret_cast<f32x4*>(&tile[(32 * wr + r) * LINE + 128 * wc + 32 * i + 2 * e + 4 * half]) =
                    f32x4{acc[i][j][e], acc[i][j][e + 1], acc[i][j][e + 2], acc[i][j][e + 3]};
        __syncthreads();
        const int n = 4 * (tid % (per / 4)), lines = 1024 / per;
        for (int row = tid / (per / 4); row < 64; row += lines) {
            const f32x4 z = *reinterpret_cast<const f32x4*>(&tile[row * LINE + n]);
            f32x4 up = {0, 0, 0, 0};
            if (a.gated) up = *reinterpret_cast<const f32x4*>(&tile[row * LINE + BIG_N / 2 + n]);
            finish4<F16>(a, m0 + 64 * (row >> 5) + 32 * j + (row & 31), n0 + n, z, up, wide);
        }
    }
}

// Rows of x up to which its 16-bit values are quantized by the lanes that multiply them; above, once for all columns.
constexpr int64_t WITHIN = 32;

template <int FORM, int XT, bool F16>
hipError_t launch_few(const MxLinearArgs& a, hipStream_t st) {
    if (a.M <= 16) return few<FORM, XT, F16, 1, 2, 16>(a, st);
    return few<FORM, XT, F16, 2, 4, 8>(a, st);
}

template <int FORM, bool F16>
hipError_t launch_type(const MxLinearArgs& a, hipStream_t st) {
    const int64_t rt = (a.M + BIG_M - 1) / BIG_M, ct = (a.out + (a.gated ? BIG_N / 2 : BIG_N) - 1) / (a.gated ? BIG_N / 2 : BIG_N);
    if (a.xs && rt * ct >= 64) {
        hipLaunchKernelGGL((many_rows_mx<FORM, F16>), dim3((unsigned)(rt * ct)), dim3(256), 0, st, a, (int)rt, (int)ct);
        return hipGetLastError();
    }
    if (a.xs) return launch_few<FORM, X_CODES, F16>(a, st);
    return launch_few<FORM, F16 ? X_F16 : X_BF16, F16>(a, st);
}

// Codes of the rows in the workspace, then their scales.
int64_t code_row(int64_t in, int form) { return form == MXFP4 ? in / 2 : in; }

}  // namespace

int64_t mx_linear_ws(int64_t M, int64_t out, int64_t in, int gated, int form, bool codes) {
    return codes || M <= WITHIN ? 0 : M * (code_row(in, form) + in / MX_BLOCK);
}

hipError_t launch_mx_linear(const MxLinearArgs& args, hipStream_t st) {
    MxLinearArgs a = args;
    if (!a.xs && a.M > WITHIN) {
        MxRowsArgs q{};
        q.values = const_cast<void*>(a.x);
        q.rows = a.M; q.len = a.in; q.ldx = a.ldx; q.ldc = code_row(a.in, a.form); q.lds = a.in / MX_BLOCK;
        q.codes = a.work; q.scales = a.work + a.M * q.ldc; q.form = a.form; q.type = a.f16;
        const hipError_t e = launch_mx_rows(q, false, st);
        if (e != hipSuccess) return e;
        a.x = q.codes; a.xs = q.scales; a.ldx = q.ldc; a.ldxs = q.lds;
    }
    if (a.form == MXFP4) return a.f16 ? launch_type<MXFP4, true>(a, st) : launch_type<MXFP4, false>(a, st);
    return a.f16 ? launch_type<MXFP8, true>(a, st) : launch_type<MXFP8, false>(a, st);
}

}  // namespace cqk
