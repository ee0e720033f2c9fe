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
#include <type_traits>

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
// of the other half), its W waves a W-th of k each; their sums join in LDS in the order of the waves.  Weights and
// x go straight into the lanes that multiply them.  x of 16 bits is quantized there, each block by the lane, or
// the two lanes, that hold it.  What it takes is a launch and a wave's chain of loads, two or four steps of them on their way
// at a time: in graphs, 1 row 3584 -> 1024 5.4 us (MXFP8 6.7; 1.9 MB), 16 rows 1024 -> 2 x 3584 4.7 (5.0), codes of 16 rows 4096
// -> 16,384 9.5 (11.0; 36 MB, 3.8 TB/s), codes of 203 rows 4096 -> 809 7.9 (10.4).
enum { X_BF16 = 0, X_F16 = 1, X_CODES = 2 };

// A row tile's x operand of 128 k: what is loaded, and what the matrix cores take.
template <int FORM, int XT>
struct XPart {
    uint4 v[XT == X_CODES ? (FORM == MXFP4 ? 1 : 2) : 4];
    __device__ __forceinline__ void load(const MxLinearArgs& a, int64_t m, int step, int quad) {
        if constexpr (XT == X_CODES) {
            const uint8_t* x = static_cast<const uint8_t*>(a.x) + m * a.ldx;
            if constexpr (FORM == MXFP4) {
                v[0] = *reinterpret_cast<const uint4*>(x + (int64_t)step * 64 + 16 * quad);
            } else {
                v[0] = *reinterpret_cast<const uint4*>(x + (int64_t)step * 128 + 16 * quad);
                v[1] = *reinterpret_cast<const uint4*>(x + (int64_t)step * 128 + 64 + 16 * quad);
            }
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
    // scale: of codes in, of values out
    __device__ __forceinline__ i32x8 take(int quad, int& scale) const {
        constexpr bool F16 = XT == X_F16;
        if constexpr (XT == X_CODES) {
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
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), col = lane & 15, quad = lane >> 4;
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
        sp[t] = a.ws + c * (a.in / MX_BLOCK);
    }
    int64_t row[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int64_t m = m0 + 16 * i + col;
        row[i] = m < a.M ? m : a.M - 1;
    }
    const int steps = (int)(a.in / 128);
    // The wave's steps [s0, s1), AHEAD of them on their way at a time.  ALWAYS: also past the end (the last one again), so that
    // the compiler knows how many loads a wait may leave.  Smaller tiles lose more by the loads; us (MXFP4
    // codes), without | with: 16 rows 5120 -> 4096 (tiles 1x2) 7.2 | 8.9, 32 rows 4096 -> 16,384 (1x4) 18.5 | 11.8, 128 rows 4096
    // -> 4096 (2x4) 15.2 | 11.3.
    const int per_wave = (steps + W - 1) / W, s0 = wave * per_wave, s1 = min(steps, s0 + per_wave);
    constexpr int AHEAD = XT == X_CODES && CT + MT * (FORM == MXFP4 ? 1 : 2) <= 8 ? 4 : 2;
    constexpr bool ALWAYS = MT * CT > 2;
    uint4 w[AHEAD][CT];
    XPart<FORM, XT> x[AHEAD][MT];
    auto fetch = [&](int j, int s) {
#pragma unroll
        for (int t = 0; t < CT; ++t) w[j][t] = *reinterpret_cast<const uint4*>(wp[t] + (int64_t)s * 64);
#pragma unroll
        for (int i = 0; i < MT; ++i) x[j][i].load(a, row[i], s, quad);
    };
    // Scales of AHEAD steps at a time, those of step s + i as a dword of the lanes of quad i.  A byte a lane for each step
    // touches as many lines as its codes and took a third of the time: 203 rows 4096 -> 809 9.9 us in place of 7.9.
    uint32_t next[CT + MT];
    auto fetch_scales = [&](int s) {
        const int64_t at = 4 * (int64_t)min(s + quad % AHEAD, steps - 1);
#pragma unroll
        for (int t = 0; t < CT; ++t) next[t] = *reinterpret_cast<const uint32_t*>(sp[t] + at);
#pragma unroll
        for (int i = 0; i < MT; ++i) next[CT + i] = XT == X_CODES ? *reinterpret_cast<const uint32_t*>(a.xs + row[i] * a.ldxs + at) : 0;
    };
    f32x4 acc[MT][CT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int t = 0; t < CT; ++t) acc[i][t] = f32x4{0, 0, 0, 0};
    auto multiply = [&](int j, const uint32_t* scales) {
        auto scale = [&](uint32_t v) { return (int)((uint32_t)__builtin_amdgcn_ds_bpermute(4 * (col + 16 * j), (int)v) >> (8 * quad)); };
        int ws[CT];
#pragma unroll
        for (int t = 0; t < CT; ++t) ws[t] = scale(scales[t]);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            int xs = XT == X_CODES ? scale(scales[CT + i]) : 0;
            const i32x8 b = x[j][i].take(quad, xs);
#pragma unroll
            for (int t = 0; t < CT; ++t) acc[i][t] = add_products<FORM>(operand(w[j][t]), ws[t], b, xs, acc[i][t]);
        }
    };
    if (s0 < s1) {
        uint32_t scales[CT + MT];
        fetch_scales(s0);
#pragma unroll
        for (int j = 0; j < AHEAD; ++j)
            if (s0 + j < s1) fetch(j, s0 + j);
        int s = s0;
        for (; s + AHEAD < s1; s += AHEAD) {
#pragma unroll
            for (int i = 0; i < CT + MT; ++i) scales[i] = next[i];
            fetch_scales(s + AHEAD);
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) {
                multiply(j, scales);
                if (ALWAYS || s + AHEAD + j < s1) fetch(j, min(s + AHEAD + j, s1 - 1));
            }
        }
#pragma unroll
        for (int j = 0; j < AHEAD; ++j)
            if (s + j < s1) multiply(j, next);
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
// Many rows: a workgroup takes BM rows of x's codes and BIG_N rows of W (gated: half of them of the gate, the others of the
// other half), KB of k a step; its waves 64 by 128 each, as 2 x 4 products of 32 x 32.  Codes and scales go from memory
// straight into LDS, STAGES - 1 steps ahead, one barrier a step.  16-byte pieces of a row lie turned in it by the row's
// number, so that the rows which a quarter of a wave reads at once are in different banks.
//
// 8192 x 4096 x 4096, codes of x given: MXFP4 86 us (3.2 PFLOP/s; a library product of bf16 matrices 195 to 213), 95 with
// bias and residual; MXFP8 189 to 203 (1.4), its operands going in twice.  The steps run at 4.6 (1.6) PFLOP/s: with neither
// loads nor reads of LDS the products alone, issued from the waves with a barrier a step, reach 6.3 (2.2).  Of the 86 us 27 are
// no steps: twice a tile's first loads and its outputs, 67 MB that all CUs write at the same time.  Residual and outputs
// past the caches (nontemporal): the same within 2 us.
constexpr int BIG_N = 256;

// The turn of a row of BYTES bytes in LDS: 16 rows read at one piece fall into all 64 banks.
template <int BYTES>
__device__ __forceinline__ int turn_of(int row) {
    return BYTES == 64 ? (row >> 2) & 3 : (row >> 1) & 7;
}
// acc += W x, 32 by 32 over 64 of k, with the scales' byte 0, or (`high`) 2.  x of MXFP8: its elements below 2, and `large`.
template <int FORM, typename X>
__device__ __forceinline__ f32x16 add_products_32(uint4 w, int ws, X x, X large, int xs, f32x16 acc, bool high) {
    const i32x8 a = operand(w);
    if constexpr (FORM == MXFP4) {
        const i32x8 b = operand(x);
        if (high) return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, acc, 4, 4, 2, ws, 2, xs);
        return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, acc, 4, 4, 0, ws, 0, xs);
    } else if (high) {
        acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, x, acc, 4, 0, 2, ws, 2, xs);
        return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, large, acc, 4, 0, 2, ws, 2, xs);
    } else {
        acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, x, acc, 4, 0, 0, ws, 0, xs);
        return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, large, acc, 4, 0, 0, ws, 0, xs);
    }
}

// WHOLE: the scales of 512 of k of a row are 16 aligned bytes.
template <int FORM, bool F16, bool WHOLE, int BM, int KB, int STAGES>
__global__ __launch_bounds__(2 * BM, 2) void many_rows_mx(MxLinearArgs a, int row_tiles, int col_tiles) {
    constexpr int WAVES = BM / 32, THREADS = 64 * WAVES, KS = KB / 64;
    constexpr int W_ROW = KB / 2, X_ROW = FORM == MXFP4 ? KB / 2 : KB;  // bytes of a step's row
    static_assert((W_ROW == 64 || W_ROW == 128) && (X_ROW == 64 || X_ROW == 128), "");
    constexpr int W_LOADS = BIG_N * W_ROW / 1024 / WAVES, X_LOADS = BM * X_ROW / 1024 / WAVES;  // a wave's a step
    constexpr int LINE = BIG_N + 4;                                                            // floats of a row in the epilogue
    struct Stage {
        uint8_t w[BIG_N * W_ROW], x[BM * X_ROW];
    };
    constexpr int PASS = BM / 2;  // rows of the epilogue at a time
    constexpr int BYTES = STAGES * sizeof(Stage) > PASS * LINE * 4 ? STAGES * sizeof(Stage) : PASS * LINE * 4;
    // Scales, four dwords (512 of k) of a row at a time, those of x behind those of W.  MXFP8: two sets, read step by step;
    // MXFP4: one, taken into registers.
    constexpr int ROWS = BIG_N + BM, SET = 4 * ROWS, SETS = FORM == MXFP4 ? 1 : 2, CHUNK = 512 / KB;  // (steps)
    __shared__ struct {
        __align__(1024) uint32_t scales[SETS * SET];  // (in front: their offsets are constants of the reads)
        __align__(1024) uint8_t stages[BYTES];
    } lds;
    uint32_t* scales_of = lds.scales;
    Stage* stage = reinterpret_cast<Stage*>(lds.stages);
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 31, half = lane >> 5, wr = wave % (BM / 64), wc = wave / (BM / 64);
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
    const int64_t m0 = rt * BM, n0 = ct * per;
    // row of W for row i of the tile; past the edge the last one
    auto w_row = [&](int i) {
        const bool up = a.gated && i >= BIG_N / 2;
        const int64_t o = n0 + (up ? i - BIG_N / 2 : i);
        return (o < a.out ? o : a.out - 1) + (up ? a.out : 0);
    };
    auto x_row = [&](int i) { return m0 + i < a.M ? m0 + i : a.M - 1; };
    const int steps = (int)(a.in / KB), dwords = (int)(a.in / 128);
    // a lane's pieces of the tile, as offsets from its first row (a wave's rows of W are all in one half)
    const int w_first = BIG_N / WAVES * wave, x_first = BM / WAVES * wave;
    const uint8_t* w_base = a.w + (n0 + (a.gated && w_first >= BIG_N / 2 ? a.out : 0)) * (a.in / 2);
    const uint8_t* x_base = static_cast<const uint8_t*>(a.x) + m0 * a.ldx;
    uint32_t w_at[W_LOADS], x_at[X_LOADS];
#pragma unroll
    for (int i = 0; i < W_LOADS; ++i) {
        const int row = w_first + 1024 / W_ROW * i + lane / (W_ROW / 16), o = a.gated ? row % (BIG_N / 2) : row;
        w_at[i] = (uint32_t)(n0 + o < a.out ? o : a.out - 1 - n0) * (uint32_t)(a.in / 2) + 16 * (lane % (W_ROW / 16) ^ turn_of<W_ROW>(row));
    }
#pragma unroll
    for (int i = 0; i < X_LOADS; ++i) {
        const int row = x_first + 1024 / X_ROW * i + lane / (X_ROW / 16);
        x_at[i] = (uint32_t)(x_row(row) - m0) * (uint32_t)a.ldx + 16 * (lane % (X_ROW / 16) ^ turn_of<X_ROW>(row));
    }
    // Scales go 16 bytes a row where they lie so, else as a dword of every 128 of k, [128 of k][row].
    constexpr int GROUPS = ROWS / 64, SHARES = (GROUPS + WAVES - 1) / WAVES;
    const uint8_t* sp[SHARES];
#pragma unroll
    for (int i = 0; i < SHARES; ++i) {
        const int row = 64 * (wave + WAVES * i) + lane;
        sp[i] = row < BIG_N ? a.ws + w_row(row) * (a.in / MX_BLOCK) : a.xs + x_row(row - BIG_N) * a.ldxs;
    }
    auto ask_scales = [&](int chunk) {  // past the last one: that one again, where nothing reads it
        const int q = 4 * chunk < dwords ? 4 * chunk : (dwords - 1) & ~3;
        uint32_t* to = scales_of + (SETS == 2 ? chunk % 2 * SET : 0);
#pragma unroll
        for (int i = 0; i < SHARES; ++i) {
            const int group = wave + WAVES * i;
            if (GROUPS % WAVES && group >= GROUPS) break;
            if constexpr (WHOLE) {
                load_to_lds(sp[i] + 4 * q, to + 256 * group);
            } else {
#pragma unroll
                for (int x = 0; x < 4; ++x) load_to_lds_4(sp[i] + 4 * (q + x < dwords ? q + x : dwords - 1), to + x * ROWS + 64 * group);
            }
        }
    };
    constexpr int SCALE_LOADS = WHOLE ? 1 : 4;  // a wave's, at least
    // Scales of the lane's rows: of a whole chunk (MXFP4), of step s (MXFP8); `held` are those of the step in hand, the
    // lane's own blocks at the bottom.
    uint32_t scales[6][SETS == 1 ? 4 : 1], held[6];
    auto take_scales = [&](int s) {
        const uint32_t* from = scales_of + (SETS == 2 ? s / CHUNK % 2 * SET : 0);
#pragma unroll
        for (int i = 0; i < 6; ++i) {
            const int row = i < 4 ? 128 * wc + 32 * i + r : BIG_N + 64 * wr + 32 * (i - 4) + r;
            if constexpr (SETS == 2) {
                scales[i][0] = WHOLE ? from[4 * row + s % 4] : from[s % 4 * ROWS + row];
            } else if constexpr (WHOLE) {
                const uint4 v = *reinterpret_cast<const uint4*>(from + 4 * row);
                scales[i][0] = v.x, scales[i][1] = v.y, scales[i][2] = v.z, scales[i][3] = v.w;
            } else {
#pragma unroll
                for (int x = 0; x < 4; ++x) scales[i][x] = from[x * ROWS + row];
            }
        }
    };
    constexpr int LOADS = W_LOADS + X_LOADS;
    // load i of step k (past the last one: that one again, where nothing reads it) into place b
    auto ask_one = [&](int k, int b, int i) {
        Stage& t = stage[b];
        const int64_t at = k < steps ? k : steps - 1;
        if (i < W_LOADS) load_to_lds(w_base + at * W_ROW, w_at[i], &t.w[W_ROW * w_first + 1024 * i]);
        else load_to_lds(x_base + at * X_ROW, x_at[i - W_LOADS], &t.x[X_ROW * x_first + 1024 * (i - W_LOADS)]);
    };
    f32x16 acc[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
    // Operands of the 64 of k in hand.  A register is read again, for the next 64, as soon as its last product is issued.
    // MXFP4: the products go by W's rows, and x, of which all is needed to the end, is read into `next`.  MXFP8: they go by
    // x's rows, which take twice the registers and are split; the second is read beside the first one's products.
    constexpr bool BY_X = FORM == MXFP8;
    uint4 w[4];
    typedef typename std::conditional<FORM == MXFP4, uint4, i32x8>::type X;
    X x[2], large[2], next[BY_X ? 1 : 2];
    auto read_w = [&](int i, int b, int ks) {
        w[i] = *reinterpret_cast<const uint4*>(
            &stage[b].w[(128 * wc + 32 * i + r) * W_ROW + 16 * ((2 * ks + half) ^ turn_of<W_ROW>(r))]);
    };
    auto read_x = [&](X& to, int j, int b, int ks) {
        const uint8_t* row = &stage[b].x[(64 * wr + 32 * j + r) * X_ROW];
        if constexpr (FORM == MXFP4)
            to = *reinterpret_cast<const uint4*>(row + 16 * ((2 * ks + half) ^ turn_of<X_ROW>(r)));
        else
            to = operand(*reinterpret_cast<const uint4*>(row + 16 * ((4 * ks + half) ^ turn_of<X_ROW>(r))),
                         *reinterpret_cast<const uint4*>(row + 16 * ((4 * ks + 2 + half) ^ turn_of<X_ROW>(r))));
    };
    ask_scales(0);
#pragma unroll
    for (int s = 0; s < STAGES; ++s)
#pragma unroll
        for (int i = 0; i < LOADS; ++i) ask_one(s, s, i);
    loaded_and_read<(STAGES - 1) * LOADS>();
    take_scales(0);
#pragma unroll
    for (int j = 0; j < (BY_X ? 1 : 2); ++j) read_x(BY_X ? x[0] : next[j], j, 0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) read_w(i, 0, 0);
    // Step by step.  The barrier stands in the last 64 of k of a step, whose operands are in registers: behind it the next
    // step's codes are read, and this step's place in LDS is asked for again, one load in a slot (all in a row they hold
    // the wave up), those left over in front of the next barrier.
    constexpr int APART = 8 * KS / LOADS;
    constexpr int UNROLL = SETS == 1 ? CHUNK : 1;  // (a chunk's scales are in registers, by number)
    int here = 0, before = STAGES - 1;             // places of this step and of the one before
    for (int s0 = 0; s0 < steps; s0 += UNROLL) {
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const int s = s0 + u, c = SETS == 1 ? u : s % CHUNK;
            if (u > 0 && s >= steps) break;
            const int after = here + 1 < STAGES ? here + 1 : 0;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                if (SETS == 2 ? ks == 0 : ks % 2 == 0)
#pragma unroll
                    for (int i = 0; i < 6; ++i) held[i] = scales[i][SETS == 1 ? u * (KB / 128) + ks / 2 : 0] >> (8 * half);
                if constexpr (!BY_X)
#pragma unroll
                    for (int j = 0; j < 2; ++j) x[j] = large[j] = next[j];
                const bool last = ks == KS - 1;
#pragma unroll
                for (int slot = 0; slot < 8; ++slot) {
                    const int i = BY_X ? slot % 4 : slot / 2, j = BY_X ? slot / 4 : slot % 2;
                    if constexpr (BY_X)
                        if (i == 0) {
                            large[j] = large_elements(x[j]);
                            x[j] ^= large[j];
                        }
                    acc[i][j] = add_products_32<FORM>(w[i], (int)held[i], x[j], large[j], (int)held[4 + j], acc[i][j], ks % 2);
                    if (last && slot == 1) {
                        // the next step's codes are needed, those behind them and scales asked for since may be on their way
                        if (STAGES == 3 && c == 1) loaded_and_read<(STAGES - 2) * LOADS + SCALE_LOADS>();
                        else loaded_and_read<(STAGES - 2) * LOADS>();
                        if (c == 0) ask_scales(s / CHUNK + 1);
                        if (SETS == 2 || c == CHUNK - 1) take_scales(s + 1);
                    }
                    const int from = last ? after : here, from_ks = last ? 0 : ks + 1;
                    if constexpr (BY_X) {
                        if (slot == 0) read_x(x[1], 1, here, ks);
                        if (slot == 3) read_x(x[0], 0, from, from_ks);
                    } else if (slot == 1 || slot == 2) {
                        read_x(next[slot - 1], slot - 1, from, from_ks);
                    }
                    if (j == 1) read_w(i, from, from_ks);
                    // slots since the barrier, this step's or the one before's (in the first step: loads done already)
                    const bool since = last && slot >= 2;
                    const int at = since ? slot - 2 : 6 + 8 * ks + slot;
                    if (at % APART == 0 && at / APART < LOADS) ask_one(since ? s + STAGES : s + STAGES - 1, since ? here : before, at / APART);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            before = here;
            here = after;
        }
    }
    loaded_to_lds();  // what was asked for past the end
    // The epilogue, 32 rows of every wave at a time through LDS: a thread then has eight neighbouring outputs of a row at a
    // time, at the same columns, and residual and y move in whole lines.
    float* tile = reinterpret_cast<float*>(lds.stages);  // [PASS][LINE]
    const bool wide = outputs_in_eights(a);
    const int n = 8 * (tid % (per / 8));
    const bool there = n0 + n < a.out;
    const int64_t o = there ? n0 + n : a.out - 8;
    float bias[8] = {}, up_bias[8] = {};
    if (wide && a.bias) {
        eight<F16>(*reinterpret_cast<const uint4*>(a.bias + o), bias);
        if (a.gated) eight<F16>(*reinterpret_cast<const uint4*>(a.bias + a.out + o), up_bias);
    }
    // a thread's rows, four at a time, every `apart`-th
    const int apart = THREADS / (per / 8);
    Residuals<4> now, next_rows;
#pragma unroll 1
    for (int j = 0; j < 2; ++j) {
        auto row_at = [&](int row) { return m0 + 64 * (row >> 5) + 32 * j + (row & 31); };
        auto row_of = [&](int i) { return row_at(apart * i + tid / (per / 8)); };
        if (wide) now.ask(a, o, row_of);
        __syncthreads();
#pragma unroll
        for (int jj = 0; jj < 2; ++jj)
            if (j == jj)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int e = 0; e < 16; e += 4)
                        *reinterpret_cast<f32x4*>(&tile[(32 * wr + r) * LINE + 128 * wc + 32 * i + 2 * e + 4 * half]) =
                            f32x4{acc[i][jj][e], acc[i][jj][e + 1], acc[i][jj][e + 2], acc[i][jj][e + 3]};
        __syncthreads();
        if (!wide) {
            const int c = tid & (per - 1);
            if (n0 + c < a.out)
#pragma unroll 1
                for (int row = tid / per; row < PASS && row_at(row) < a.M; row += THREADS / per)
                    finish<F16>(a, row_at(row), n0 + c, tile[row * LINE + c], a.gated ? tile[row * LINE + BIG_N / 2 + c] : 0.0f);
            continue;
        }
#pragma unroll 1
        for (int i0 = 0; i0 < PASS / apart; i0 += 4) {
            if (i0 + 4 < PASS / apart) next_rows.ask(a, o, [&](int i) { return row_of(i0 + 4 + i); });
            if (there)
                finish8<F16, BIG_N / 2, 4>(
                    a, o, bias, up_bias, now, [&](int i) { return row_of(i0 + i); },
                    [&](int i) {
                        return (const __attribute__((address_space(3))) float*)&tile[(apart * (i0 + i) + tid / (per / 8)) * LINE + n];
                    });
            now = next_rows;
        }
    }
}

template <int FORM, bool F16, int BM, int KB, int STAGES>
hipError_t many(const MxLinearArgs& a, hipStream_t st) {
    if (a.in % KB != 0) return hipErrorInvalidValue;  // (a kernel of whole steps: what is left would be lost, or read in front of k)
    const int per = a.gated ? BIG_N / 2 : BIG_N;
    const int64_t rt = (a.M + BM - 1) / BM, ct = (a.out + per - 1) / per;
    const dim3 grid((unsigned)(rt * ct));
    if (a.in % 512 == 0 && a.ldxs % 16 == 0 && ((uintptr_t)a.ws | (uintptr_t)a.xs) % 16 == 0)
        hipLaunchKernelGGL((many_rows_mx<FORM, F16, true, BM, KB, STAGES>), grid, dim3(2 * BM), 0, st, a, (int)rt, (int)ct);
    else
        hipLaunchKernelGGL((many_rows_mx<FORM, F16, false, BM, KB, STAGES>), grid, dim3(2 * BM), 0, st, a, (int)rt, (int)ct);
    return hipGetLastError();
}

int64_t up(int64_t n, int64_t of) { return (n + of - 1) / of; }

// Whether x's 16-bit values are quantized by the lanes that multiply them (again for every tile of columns), or once,
// before.  us in graphs, within | before (some 2 of them the other launch): 16 rows, 1024 -> 2 x 3584 4.7 | 6.7, 4096 ->
// 4096 8.9 | 7.9 (MXFP8 9.5 | 9.1; called from Python 9.0 | 11.6, for the workspace and the launch), 4096 -> 16,384 12.7 | 11.8
// (15.3 | 13.3); 32 rows, 4096 -> 4096 8.9 | 8.7, 4096 -> 16,384 18.4 | 14.4; 64 rows, 3584 -> 1024 7.6 | 7.9, 4096 -> 4096
// 13.6 | 10.4.  Through more than 16,384 columns, MXFP8: 1 row, 4096 -> 41,024 28.3 | 28.4, 4 rows 30.3 | 29.5, 8 rows 33.2 | 30.6,
// 16 rows 42.5 | 33.7, 4096 -> 128,256 114 | 85, 1024 -> 41,024 16.6 | 16.7; MXFP4, whose conversion is half as long: 16 rows,
// 4096 -> 41,024 31.1 | 29.6, 1024 -> 41,024 11.7 | 15.5.
bool within(int64_t M, int64_t cols, int form) {
    if (M <= 16) return form == MXFP4 || M <= 4 || up(cols, 64) <= 256;
    return M <= 64 && up(M, 16) * up(cols, 64) <= 128;
}

// The smallest tile of rows and columns, and with it the most waves to a sum, with which the workgroups fit on the chip's 256
// CUs at once: they take the time of their own chain of loads, and another round of them takes it again.  us, by rows and
// columns of a tile in 16s:
//                                     1x2     2x2     1x4     2x4     4x4
//   1 row, 4096 -> 4096               6.2             9.1                    (16-bit x, MXFP4)
//   16 rows, 1024 -> 2 x 3584         4.8             5.8
//   203 rows, 4096 -> 809            10.7     7.9     9.2    11.2    17.4    (codes)
//   128 rows, 4096 -> 4096           20.3    12.2    17.1    11.3    17.4
//   1024 rows, 3584 -> 1024          33.5    17.4    28.2    18.5    16.6
//   64 rows, 4096 -> 16,384          40.7    21.4    33.7    21.9    17.9
// 8 waves a tile (4x4: 4); 16 in place of 8 are as fast or slower up to 0.5 us.
template <int FORM, int XT, bool F16>
hipError_t launch_few(const MxLinearArgs& a, hipStream_t st) {
    const int64_t cols = a.gated ? 2 * a.out : a.out;
    if (up(a.M, 16) * up(cols, 32) <= 256) return few<FORM, XT, F16, 1, 2, 8>(a, st);
    if constexpr (XT == X_CODES) {
        if (up(a.M, 32) * up(cols, 32) <= 256 && a.M > 16) return few<FORM, XT, F16, 2, 2, 8>(a, st);
        if (up(a.M, 16) * up(cols, 64) <= 256 || a.M <= 16) return few<FORM, XT, F16, 1, 4, 8>(a, st);
        if (up(a.M, 32) * up(cols, 64) <= 256) return few<FORM, XT, F16, 2, 4, 8>(a, st);
        return few<FORM, XT, F16, 4, 4, 4>(a, st);
    } else {  // (at most 16 rows: see within)
        return few<FORM, XT, F16, 1, 4, 8>(a, st);
    }
}

template <int FORM, bool F16>
hipError_t launch_type(const MxLinearArgs& a, hipStream_t st) {
    if (!a.xs) return launch_few<FORM, F16 ? X_F16 : X_BF16, F16>(a, st);
    const int64_t cols = a.gated ? 2 * a.out : a.out;
    // Where tiles of 64 by 64 no longer fit on the chip at once, the other kernel reads operands once for more products; with
    // MXFP8, which takes its steps four times as long, from two rounds and a half of them on.  us, few | many: MXFP4 64 rows,
    // 4096 -> 16,384 17.9 | 22.1, 512 rows, 4096 -> 4096 36 | 22; MXFP8 512 rows 44 | 55, 1024 rows 78 | 63, 203 rows,
    // 4096 -> 16,384 70 | 63, 512 rows, 1024 -> 2 x 3584 31 | 21.  Few rows stay with tiles of 16 of them whatever the columns,
    // of which the other kernel would multiply 128: 1 row, 4096 -> 24,576 MXFP4 14.7 | 21.0, 4096 -> 41,024 23.0 | 22.7 (MXFP8
    // 26 | 62), 4096 -> 128,256 61 | 73 (69 | 102); 8 rows, 4096 -> 41,024 24.9 | 24.0 (28 | 62), 1024 -> 128,256 31.6 | 32.0
    // (34.1 | 32.5); 16 rows MXFP4 17.6 | 21.8, 27.2 | 24.6 and, 1024 -> 128,256, 35.7 | 32.7, MXFP8 31 | 63, 82 | 106 and 38.6 |
    // 33.1.
    if (up(a.M, 64) * up(cols, 64) <= (FORM == MXFP4 ? 256 : 640) || a.M <= (FORM == MXFP4 ? 8 : 16))
        return launch_few<FORM, X_CODES, F16>(a, st);
    if constexpr (FORM == MXFP4) {
        // 256 rows a workgroup and 256 of k a step, one workgroup a CU, where that leaves few CUs idle; us, 128 rows | 256:
        // 2048 x 4096 x 4096 30.5 | 34.7, 2048 x 2 x 3584 x 1024 22.1 | 20.6, 4096 x 4096 x 4096 52 | 43, 4096 x 16,384 x
        // 4096 189 | 159.
        if (a.in % 256 == 0 && up(a.M, 256) * up(cols, 256) >= 192) return many<MXFP4, F16, 256, 256, 2>(a, st);
        return many<MXFP4, F16, 128, 128, 3>(a, st);
    } else {
        // (256 rows a workgroup: between 5 % faster and 3 % slower, by the shape)
        return many<MXFP8, F16, 128, 128, 2>(a, st);
    }
}

// Codes of the rows in the workspace, then their scales.
int64_t code_row(int64_t in, int form) { return form == MXFP4 ? in / 2 : in; }

}  // namespace

int64_t mx_linear_ws(int64_t M, int64_t out, int64_t in, int gated, int form, bool codes) {
    return codes || within(M, gated ? 2 * out : out, form) ? 0 : M * (code_row(in, form) + in / MX_BLOCK);
}

hipError_t launch_mx_linear(const MxLinearArgs& args, hipStream_t st) {
    MxLinearArgs a = args;
    if (!a.xs && !within(a.M, a.gated ? 2 * a.out : a.out, a.form)) {
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
