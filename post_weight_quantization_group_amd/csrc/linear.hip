// Linear layer over GPTQ-v1 tensors with its epilogue, for gfx950:
//
//   z[m][c] = sum_g s[g][c] sum_{k in g} x[m][k] (u[k][c] - 8),    y = act(z + b) [* (z' + b')] + r.
//
// The products run on the matrix cores, in x's own 16-bit type: the codes u - 8 are exact in both,
// so are their products with x in fp32, and the sums are fp32.  A qweight word holds eight
// consecutive k of one column, which is what one lane of the B operand takes: words are dequantized in the
// registers of the lane that multiplies them.
//
// Lane layouts (checked on gfx950).  16x16x32: lane l holds A[l % 16][8 (l / 16) + e], B[8 (l / 16) +
// e][l % 16], D[4 (l / 16) + r][l % 16].  32x32x16: A[l % 32][8 (l / 32) + e], B likewise,
// D[8 (r / 4) + 4 (l / 32) + r % 4][l % 32].
#include "epilogue.h"
#include "serve_args.h"
#include "serve_math.h"

namespace cqk {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

template <bool F16>
__device__ __forceinline__ f32x4 mfma16(uint4 a, uint4 b, f32x4 c) {
    if constexpr (F16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
template <bool F16>
__device__ __forceinline__ f32x16 mfma32(uint4 a, uint4 b, f32x16 c) {
    if constexpr (F16)
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// The eight codes of a word as 16 (u - 8) in the 16-bit type: u XOR 8 is u - 8 as a signed 4-bit
// field, which in the upper half of a byte reads as 16 times its value, converted by one
// instruction per code (a byte's conversion with sign extension); exact in both types, and the 1/16
// goes into the group's scale.  15 instructions a word against 21 with the fields shifted down.  A mask of
// 0 in place of FIELDS makes the codes 0.
constexpr float CODE_UNIT = 1.0f / 16.0f;
constexpr uint32_t FIELDS = 0xF0F0F0F0u;
__device__ __forceinline__ uint32_t even_codes(uint32_t word, uint32_t mask) { return ((word << 4) ^ 0x80808080u) & mask; }
__device__ __forceinline__ uint32_t odd_codes(uint32_t word, uint32_t mask) { return (word ^ 0x88888888u) & mask; }
// Codes 2 j and 2 j + 1.
template <bool F16>
__device__ __forceinline__ uint32_t two_codes(uint32_t even, uint32_t odd, int j) {
    const float lo = (float)(int8_t)(even >> (8 * j)), hi = (float)(int8_t)(odd >> (8 * j));
    if constexpr (F16) return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(lo, hi));
    return __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
}
template <bool F16>
__device__ __forceinline__ uint4 codes(uint32_t word) {
    const uint32_t even = even_codes(word, FIELDS), odd = odd_codes(word, FIELDS);
    return make_uint4(two_codes<F16>(even, odd, 0), two_codes<F16>(even, odd, 1), two_codes<F16>(even, odd, 2),
                      two_codes<F16>(even, odd, 3));
}

__device__ __forceinline__ float scale_of(uint16_t bits) { return (float)__builtin_bit_cast(_Float16, bits); }

// ---------------------------------------------------------------------------------------------
// Few rows, or few tiles: a workgroup takes 16 MT rows and 4 x 16 columns (gated: 2 x 16 of the gate and
// the same of the other half), its W waves every W-th group, and their sums join in LDS in the order
// of the waves.  For one row the weights' words are all there is to read, and each lane reads 16
// bytes of them at a time (VEC); x comes straight from memory, no wave needs another's.  Bound by the latency of its
// few rounds of loads: 1 row, 3584 -> 1024 8.0 us (16 waves in place of 8: 7.7); 16 rows, 1024 -> 2 x 3584 gated 5.3
// (5.5); 203 rows, 4096 -> 809 14.3.  With enough columns by the words' bytes: 1 row, 4096 -> 128,256 59 us, 4.6 TB/s.
template <bool F16, int MT, int W, bool VEC>
__global__ __launch_bounds__(64 * W) void few_rows_linear(LinearArgs a, int col_tiles) {
    __shared__ __align__(16) float sums[W * MT * 16 * 64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, col = lane & 15, quad = lane >> 4;
    const int64_t ct = blockIdx.x % col_tiles, rt = blockIdx.x / col_tiles;
    const int64_t cols = a.gated ? 2 * a.out : a.out;
    const int per = a.gated ? 32 : 64;  // outputs per workgroup
    const int64_t n0 = ct * per, m0 = rt * (16 * MT);
    // slot t of lane column `col` is output n0 + local[t] of column half[t]
    int64_t c[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const int64_t o = n0 + (VEC ? (a.gated ? 2 * col + (t & 1) : 4 * col + t) : col + 16 * (a.gated ? t & 1 : t));
        c[t] = (o < a.out ? o : a.out - 1) + (a.gated && t >= 2 ? a.out : 0);
        // (past the edge: any column in range; VEC loads whole runs of 4 or 2, which end together with it)
    }
    if (VEC) {
        const int run = a.gated ? 2 : 4;
        if (n0 + run * col >= a.out) {
#pragma unroll
            for (int t = 0; t < 4; ++t) c[t] = (a.out - run) + (t & (run - 1)) + (a.gated && t >= 2 ? a.out : 0);
        }
    }
    const uint16_t* xrow[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int64_t m = m0 + 16 * i + col;
        xrow[i] = a.x + (m < a.M ? m : a.M - 1) * a.ldx + 8 * quad;
    }
    const int groups = (int)(a.in / 128);
    uint32_t wr[4][4];  // [k step][slot]
    uint4 xr[MT][4];
    float sc[4];
    auto fetch = [&](int g) {
        if (g >= groups) return;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            const int32_t* q = a.qw + ((int64_t)g * 16 + 4 * ks + quad) * cols;
            if (VEC && !a.gated) {
                const uint4 v = *reinterpret_cast<const uint4*>(q + c[0]);
                wr[ks][0] = v.x; wr[ks][1] = v.y; wr[ks][2] = v.z; wr[ks][3] = v.w;
            } else if (VEC) {
                const uint2 v = *reinterpret_cast<const uint2*>(q + c[0]), u = *reinterpret_cast<const uint2*>(q + c[2]);
                wr[ks][0] = v.x; wr[ks][1] = v.y; wr[ks][2] = u.x; wr[ks][3] = u.y;
            } else {
#pragma unroll
                for (int t = 0; t < 4; ++t) wr[ks][t] = (uint32_t)q[c[t]];
            }
#pragma unroll
            for (int i = 0; i < MT; ++i) xr[i][ks] = *reinterpret_cast<const uint4*>(xrow[i] + (int64_t)g * 128 + 32 * ks);
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) sc[t] = scale_of(a.scales[(int64_t)g * cols + c[t]]) * CODE_UNIT;
    };
    f32x4 acc[MT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int t = 0; t < 4; ++t) acc[i][t] = f32x4{0, 0, 0, 0};
    fetch(wave);
    for (int g = wave; g < groups; g += W) {
        f32x4 part[MT][4];
        float s[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            s[t] = sc[t];
#pragma unroll
            for (int i = 0; i < MT; ++i) part[i][t] = f32x4{0, 0, 0, 0};
        }
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const uint4 b = codes<F16>(wr[ks][t]);
#pragma unroll
                for (int i = 0; i < MT; ++i) part[i][t] = mfma16<F16>(xr[i][ks], b, part[i][t]);
            }
        fetch(g + W);
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][t][e] = __builtin_fmaf(s[t], part[i][t][e], acc[i][t][e]);
    }
    // sums[wave][row][slot * 16 + col]
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) sums[((wave * MT + i) * 16 + 4 * quad + e) * 64 + 16 * t + col] = acc[i][t][e];
    __syncthreads();
    for (int i = tid; i < MT * 16 * per; i += 64 * W) {
        const int row = i / per, n = i % per;
        const int64_t m = m0 + row, o = n0 + n;
        if (m >= a.M || o >= a.out) continue;
        int at;  // where output n of the tile lies among the 64 slots
        if (!VEC) at = n;
        else if (a.gated) at = 16 * (n & 1) + n / 2;
        else at = 16 * (n & 3) + n / 4;
        float z = 0.0f, up = 0.0f;
#pragma unroll
        for (int x = 0; x < W; ++x) {
            z += sums[(x * MT * 16 + row) * 64 + at];
            if (a.gated) up += sums[(x * MT * 16 + row) * 64 + 32 + at];
        }
        finish<F16>(a, m, o, z, up);
    }
}

// ---------------------------------------------------------------------------------------------
// Many rows: a workgroup takes 128 rows and 256 columns (gated: 128 of either half), each of its four
// waves all rows and 64 columns, as 4 x T tiles of 32 x 32 (T = 1: half the columns).  x and the qweight words go from memory
// straight into LDS, a group ahead: x, in two buffers, for all waves; the words for the wave that
// dequantizes them, which has taken them into registers before the next ones are asked for.
//
// The accumulators hold z / s_g: at a group's start they are multiplied by s_{g-1} / s_g, and the
// matrix cores add the group's products on top.  Sums per group beside them, scaled in by an fma,
// would take another 128 registers and leave one wave per SIMD instead of two.  It costs a group two more
// fp32 roundings (the ratio and its product).  A scale of 0 leaves the accumulators as they are and masks its codes to 0.
//
// A group's 64 products per wave (32 cycles each, T = 2) come with 15 instructions per word (240) and 128
// multiplications: 5.8 vector instructions a product, of which 6 run beside one for nothing where
// they stand between the products; so the order is written out, slot by slot.  8192 rows, 4096 -> 4096 bf16: 268 to 305 us by the card
// and its clock, 0.9 to 1.0 PFLOP/s (the library's product of dense bf16 matrices of these sizes 211); without the loads it took 211, so what
// bounds it is their issue between the products (all in a row: 290).
constexpr int BIG_M = 128;

// T: column tiles of a wave.  PAIR: its two columns of a lane are neighbours (not gated).  WIDE: words move 16 bytes a lane.
template <bool F16, int T, bool PAIR, bool WIDE>
__global__ __launch_bounds__(256, 2) void many_rows_linear(LinearArgs a, int row_tiles, int col_tiles) {
    __shared__ __align__(16) uint16_t xs[2][BIG_M * 128];
    constexpr int COLS = 32 * T, EACH = COLS / 2;  // columns of a wave; gated: of either half
    __shared__ __align__(16) uint32_t words[4][16 * COLS];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), col = lane & 31,
              half = lane >> 5;
    const int64_t cols = a.gated ? 2 * a.out : a.out;
    const int per = a.gated ? 4 * EACH : 4 * COLS;  // outputs per workgroup
    // Workgroups go to the eight XCDs in turn: each XCD takes a run of tiles, in bands of 8 row tiles,
    // so that the tiles it works on at a time share rows of x and columns of W in its L2.
    int64_t id = blockIdx.x;
    const int64_t all = (int64_t)row_tiles * col_tiles;
    {
        const int64_t base = all / 8, more = all % 8, x = id % 8, j = id / 8;
        id = x * base + (x < more ? x : more) + j;
    }
    const int64_t band = id / (8 * col_tiles), in_band = id % (8 * col_tiles);
    const int64_t high = row_tiles - band * 8 < 8 ? row_tiles - band * 8 : 8;
    const int64_t rt = band * 8 + in_band % high, ct = in_band / high;
    const int64_t m0 = rt * BIG_M, n0 = ct * per + wave * (per / 4);
    // Column of slot k of the wave's: gated: half of them of the gate, then the same of the other half.  Past the
    // edge: any column in range (WIDE: runs of four that start at a multiple of four, which end with it).
    auto column = [&](int k) {
        const int64_t o = n0 + (a.gated ? k & (EACH - 1) : k), edge = WIDE ? a.out - 4 + (k & 3) : a.out - 1;
        return (o < a.out ? o : edge) + (a.gated && k >= EACH ? a.out : 0);
    };
    int64_t c[T];
#pragma unroll
    for (int t = 0; t < T; ++t) c[t] = column(PAIR ? 2 * col + t : 32 * t + col);
    const int groups = (int)(a.in / 128);
    constexpr int FIRST = 2 * T, APART = T == 1 ? 2 : 3;  // slots of the loads of x

    // x tile of a group: 16-byte piece p of row r lies at place p XOR (r % 16) of its row, so that the 16
    // rows a quarter of a wave reads at once lie in different banks.  A wave's load fills 1 KB: four rows.
    const uint16_t* xp[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int row = 32 * wave + 4 * i + (lane >> 4);
        const int64_t m = m0 + row < a.M ? m0 + row : a.M - 1;
        xp[i] = a.x + m * a.ldx + 8 * ((lane & 15) ^ (row & 15));
    }
    auto ask_x = [&](int g, int i, int buf) { load_to_lds(xp[i] + (int64_t)g * 128, &xs[buf][(32 * wave + 4 * i) * 128]); };
    // words: qweight row r of the group in row r of the wave's LDS, its slots in order
    constexpr int A_LOAD = WIDE ? 256 : 64, WORD_LOADS = 16 * COLS / A_LOAD;  // words a load
    constexpr int LINE = COLS / (WIDE ? 4 : 1), LINES = 64 / LINE;  // lanes a row, rows a load
    const int32_t* wp = a.qw + lane / LINE * cols + column((WIDE ? 4 : 1) * (lane % LINE));
    auto ask_words = [&](int g, int i) {
        const int32_t* from = wp + ((int64_t)g * 16 + LINES * i) * cols;
        if constexpr (WIDE) load_to_lds(from, &words[wave][i * A_LOAD]);
        else load_to_lds_4(from, &words[wave][i * A_LOAD]);
    };
    // step ks of a group (k = 16 ks ..) takes qweight row 2 ks + half
    uint32_t w[8][T];
    auto take_words = [&] {
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
            const uint32_t* row = &words[wave][(2 * ks + half) * COLS];
            if constexpr (PAIR) {
                const uint2 v = *reinterpret_cast<const uint2*>(row + 2 * col);
                w[ks][0] = v.x; w[ks][1] = v.y;
            } else {
#pragma unroll
                for (int t = 0; t < T; ++t) w[ks][t] = row[32 * t + col];
            }
        }
    };

    f32x16 acc[4][T];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][t][e] = 0.0f;

    // Scales of the group in hand: the ratio the accumulators take on, and the mask of its codes.
    float s[T], ratio[T];
    uint32_t mask[T];
    uint16_t sn[T];
#pragma unroll
    for (int t = 0; t < T; ++t) s[t] = 1.0f;
    auto take_scales = [&] {
#pragma unroll
        for (int t = 0; t < T; ++t) {
            uint32_t bits = sn[t];
            asm volatile("" : "+v"(bits));  // the wait for it belongs here, not behind its load
            const float sg = scale_of((uint16_t)bits);
            const bool zero = sg == 0.0f;
            ratio[t] = zero ? 1.0f : s[t] / sg;
            s[t] = zero ? s[t] : sg;
            mask[t] = zero ? 0u : FIELDS;
        }
    };
    auto scale_tile = [&](int j) {
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[j / T][j % T][e] *= ratio[j % T];
    };

#pragma unroll 1
    for (int i = 0; i < WORD_LOADS; ++i) ask_words(0, i);
#pragma unroll
    for (int i = 0; i < 8; ++i) ask_x(0, i, 0);
#pragma unroll
    for (int t = 0; t < T; ++t) sn[t] = a.scales[c[t]];
    loaded_to_lds();
    take_words();
    take_scales();
    uint32_t b[T][4], bn[T][4];  // operands of this step and of the next
#pragma unroll
    for (int j = 0; j < 4 * T; ++j)
        b[j / 4][j % 4] = two_codes<F16>(even_codes(w[0][j / 4], mask[j / 4]), odd_codes(w[0][j / 4], mask[j / 4]), j % 4);
    for (int g = 0; g < groups; ++g) {
        const uint16_t* xt = xs[g & 1];
        const int next = g + 1 < groups ? g + 1 : g;  // (the last group asks for its own once more, into the idle buffer)
        __syncthreads();                              // this group's x is in LDS, and the other buffer has been read
#pragma unroll
        for (int t = 0; t < T; ++t) sn[t] = a.scales[(int64_t)next * cols + c[t]];
        if constexpr (!WIDE) {
#pragma unroll 1
            for (int i = 0; i < WORD_LOADS; ++i) ask_words(next, i);
        }
        uint4 x[4];
        auto read_x = [&](int i, int ks) {
            const int row = 32 * i + col;
            x[i] = *reinterpret_cast<const uint4*>(xt + row * 128 + 8 * ((2 * ks + half) ^ (row & 15)));
        };
#pragma unroll
        for (int i = 0; i < 4; ++i) read_x(i, 0);
        scale_tile(0);
        uint32_t even, odd, last[T];
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
            if (ks == 6) {
#pragma unroll
                for (int t = 0; t < T; ++t) last[t] = w[7][t];
                loaded_to_lds<8>();  // (x was asked for after the words)
                take_words();
            }
            if (ks == 7) take_scales();
#pragma unroll
            for (int j = 0; j < 4 * T; ++j) {
                const int i = j / T, t = j % T, slot = 4 * T * ks + j;
                acc[i][t] = mfma32<F16>(x[i], make_uint4(b[t][0], b[t][1], b[t][2], b[t][3]), acc[i][t]);
                // an operand is read as soon as its register's last product is issued, 6 slots before its own
                if (t == T - 1 && ks < 7) read_x(i, ks + 1);
                if (ks == 0 && j < 4 * T - 1) scale_tile(j + 1);
                if (j % 4 == 0) {
                    const uint32_t word = ks == 6 ? last[j / 4] : w[(ks + 1) % 8][j / 4];
                    even = even_codes(word, mask[j / 4]);
                    odd = odd_codes(word, mask[j / 4]);
                }
                bn[j / 4][j % 4] = two_codes<F16>(even, odd, j % 4);
                // The next group's loads, one in a slot: asked for in a row, they hold the wave up (1 KB keeps
                // the memory pipe for 16 cycles or more).
                if (WIDE && slot < WORD_LOADS) ask_words(next, slot);
                else if (slot >= FIRST && slot < FIRST + 8 * APART && (slot - FIRST) % APART == 0) ask_x(next, (slot - FIRST) / APART, (g + 1) & 1);
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int j = 0; j < 4 * T; ++j) b[j / 4][j % 4] = bn[j / 4][j % 4];
        }
        loaded_to_lds();
    }
    // The epilogue, 32 rows at a time through LDS: every thread then has four neighbouring outputs of a
    // row, and residual and y move in whole lines.
    const bool wide = outputs_in_fours(a);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float* tile = reinterpret_cast<float*>(xs[i & 1]);  // [32][4 COLS]
        if (i == 0) __syncthreads();                        // the last group's x has been read
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            float* to = tile + (8 * (e >> 2) + 4 * half + (e & 3)) * (4 * COLS) + COLS * wave;
            float z[T];
#pragma unroll
            for (int t = 0; t < T; ++t) z[t] = acc[i][t][e] * (s[t] * CODE_UNIT);
            if constexpr (PAIR) {
                *reinterpret_cast<float2*>(to + 2 * col) = make_float2(z[0], z[1]);
            } else {
#pragma unroll
                for (int t = 0; t < T; ++t) to[32 * t + col] = z[t];
            }
        }
        __syncthreads();
        const int n = 4 * (tid % (per / 4)), lines = 1024 / per;
        const int at = a.gated ? n / EACH * COLS + n % EACH : n;
        for (int row = tid / (per / 4); row < 32; row += lines) {
            const f32x4 z = *reinterpret_cast<const f32x4*>(tile + row * (4 * COLS) + at);
            f32x4 up = {0, 0, 0, 0};
            if (a.gated) up = *reinterpret_cast<const f32x4*>(tile + row * (4 * COLS) + at + EACH);
            finish4<F16>(a, m0 + 32 * i + row, ct * per + n, z, up, wide);
        }
    }
}

template <bool F16, int MT, int W>
hipError_t few(const LinearArgs& a, bool vec, hipStream_t st) {
    const int per = a.gated ? 32 : 64;
    const int64_t ct = (a.out + per - 1) / per, rt = (a.M + 16 * MT - 1) / (16 * MT);
    if (ct * rt > INT32_MAX) return hipErrorInvalidValue;
    const dim3 grid((unsigned)(ct * rt));
    if (vec) hipLaunchKernelGGL((few_rows_linear<F16, MT, W, true>), grid, dim3(64 * W), 0, st, a, (int)ct);
    else hipLaunchKernelGGL((few_rows_linear<F16, MT, W, false>), grid, dim3(64 * W), 0, st, a, (int)ct);
    return hipGetLastError();
}

template <bool F16, int T>
hipError_t many(const LinearArgs& a, int64_t rt, int64_t ct, hipStream_t st) {
    if (rt * ct > INT32_MAX) return hipErrorInvalidValue;
    const dim3 grid((unsigned)(rt * ct));
    const bool wide = a.out % 4 == 0 && ((uintptr_t)a.qw & 15) == 0;
    if (T == 2 && wide && !a.gated)
        hipLaunchKernelGGL((many_rows_linear<F16, T, T == 2, true>), grid, dim3(256), 0, st, a, (int)rt, (int)ct);
    else if (wide)
        hipLaunchKernelGGL((many_rows_linear<F16, T, false, true>), grid, dim3(256), 0, st, a, (int)rt, (int)ct);
    else
        hipLaunchKernelGGL((many_rows_linear<F16, T, false, false>), grid, dim3(256), 0, st, a, (int)rt, (int)ct);
    return hipGetLastError();
}

template <bool F16>
hipError_t launch_type(const LinearArgs& a, hipStream_t st) {
    const int64_t rt = (a.M + BIG_M - 1) / BIG_M, cols = a.gated ? 2 * a.out : a.out;
    const int64_t ct2 = (cols + 255) / 256, ct1 = (cols + 127) / 128;
    const bool aligned16 = ((uintptr_t)a.qw & 15) == 0;
    // Up to 32 rows the other kernel reads the words once where this one multiplies 128 rows, and is faster at any width;
    // up to 64 it reads them twice, and is faster up to 192 tiles (us, the other | 128 columns): 1 row, 4096 -> 16,384
    // 10.7 | 39, 4096 -> 2 x 14,336 17.5 | 44, 4096 -> 128,256 60 | 144 (256 columns: 131); 32 rows, 4096 -> 16,384 16 | 41,
    // 128,256 120 | 146 (134); 1024 -> 65,536 24.1 | 25.2; 64 rows, 4096 -> 24,576 43 | 45, 32,768 57 | 46; 1024 -> 24,576
    // 17.2 | 16.9.  96 rows, 4096 -> 14,592 41 | 45, 18,432 55 | 47.
    const int64_t least = a.M <= 32 ? (int64_t)1 << 22 : a.M <= 64 ? 193 : 112;  // (2^22: the grid's threads)
    // Columns a workgroup, by 128 x 128 tiles on the chip's 256 CUs (us, 256 | 128 columns): 1024 tiles (4096 x 4096, 4096
    // inputs) 128 | 138, 896 (2048 x 2 x 3584, 1024) 42.2 | 43.7; 512 (2048 x 4096, 4096) 76 | 73, 256 (1024 x 4096) 71 | 48.
    // Below, this kernel's time no longer falls and the other's does (128 columns | other kernel): 128 tiles (512 x
    // 4096, 4096) 47 | 49, (2048 x 1024, 3584) 42 | 45; 64 tiles (256 x 4096, 4096) 42 | 28, (1024 x 1024, 3584) 42 | 23.
    if (rt * ct1 >= least) return rt * ct1 > 512 ? many<F16, 2>(a, rt, ct2, st) : many<F16, 1>(a, rt, ct1, st);
    const bool vec = a.gated ? a.out % 2 == 0 && ((uintptr_t)a.qw & 7) == 0 : a.out % 4 == 0 && aligned16;
    // Rows a tile and waves: 203 rows (4096 -> 809) 14.5 us with 32 rows and 8 waves, 17.3 with 4; 1024 rows (3584 -> 1024)
    // 22.7 us with 64 rows and 4 waves, 25.1 with 32 and 8.
    if (a.M <= 16) return few<F16, 1, 8>(a, vec, st);
    if (a.M <= 256) return few<F16, 2, 8>(a, vec, st);
    return few<F16, 4, 4>(a, vec, st);
}

}  // namespace

hipError_t launch_linear(const LinearArgs& a, hipStream_t st) {
    return a.x_f16 ? launch_type<true>(a, st) : launch_type<false>(a, st);
}

}  // namespace cqk
