// Attention of new tokens over a paged cache, for gfx950.
//
// Rows are the (token, query head) pairs of one request and one key/value head: row = token i times
// G + head of the group, so that grouped heads fill a tile together and K and V are read once for
// all of them.  One pass over the keys with the running maximum and sum of the softmax.
//
// Both products run on the matrix cores with the queries as columns:
//        S^T [keys x rows] = K Q^T,        O^T [D x rows] += V^T P^T.
// A lane then holds scores of one row only (its column), so the maximum and the sum need one or two
// exchanges between lanes, and the scores' registers are the second product's B operand as they
// stand: the order of the keys inside a contraction is free as long as V^T uses the same.  V^T comes
// out of row-major V in LDS by the transposing read (ds_read_b64_tr_b16: lane 4 j + c of 16 addresses
// row j, columns 4 c ..; lane i receives column i of the four rows).
//
// Lane layouts (checked on gfx950).  32x32x16: lane l holds A[l % 32][8 (l / 32) + e], B[8 (l / 32) +
// e][l % 32], D[8 (r / 4) + 4 (l / 32) + r % 4][l % 32].  16x16x32: A[l % 16][8 (l / 16) + e], B
// likewise, D[4 (l / 16) + r][l % 16].
//
// The weights are rounded to the 16-bit type for the product with V, which the matrix cores take at 16 times the rate of
// fp32 operands; scores, maxima, sums (of the weights before that rounding) and outputs are fp32.  Their rounding is of the
// size of the output's own: relative to 64 bits the outputs are off by 2.0e-3 to 2.4e-3 (bf16; f16 2.5e-4), an fp32
// evaluation that is rounded at the end by 1.7e-3 (2.0e-4).
//
// A masked key has weight 0, and 0 times an infinity or a NaN in V would be a NaN: keys that no row
// of the tile sees are loaded as zeros, and where a tile's mask differs between its rows, what is not
// finite in its V is staged as 0 and read again, key by key, into two bits per output (an infinity of
// either sign seen; both: NaN) that are applied at the end.
//
// The cache holds 16-bit values (KIND = CACHE_16) or microscaled blocks (MXFP4, MXFP8), whose values go into the
// same products: they are exact in the 16-bit type that they were quantized from, and converted as they arrive, two an
// instruction.
#pragma once
#include "mx.h"
#include "serve_args.h"
#include "serve_math.h"

namespace cqk {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) s16x4* lds_s16x4;

// Rows of a request up to which few_rows_kernel takes it, one workgroup a part.  32 requests against 2,000 keys (32 heads
// over 8, D = 128): 32 rows 70 us there and 54 in many_rows_kernel, 64 rows 120 and 56; 4 against 8,000: 41 and 36.
constexpr int FEW = 16;
constexpr int MANY = 256;  // rows of a workgroup of many_rows_kernel

// How far (in powers of two of the weights) the maximum that the weights are taken against may stay behind the true one:
// the sums' and the weights' relative roundings are the same up to 2^8, and most steps then leave the outputs alone.
constexpr float LAG = 8.0f;
constexpr float LN2 = 0.69314718f;

template <bool F16>
__device__ __forceinline__ f32x16 mfma32(s16x8 a, s16x8 b, f32x16 c) {
    if constexpr (F16)
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
template <bool F16>
__device__ __forceinline__ f32x4 mfma16(s16x8 a, s16x8 b, f32x4 c) {
    if constexpr (F16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

template <bool F16>
__device__ __forceinline__ s16x8 pack8(const float* p) {
    s16x8 v;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = (short)from_f32<F16>(p[e]);
    return v;
}

template <bool F16>
__device__ __forceinline__ bool not_finite(uint16_t b) {
    constexpr uint16_t E = F16 ? 0x7C00 : 0x7F80;
    return (b & E) == E;
}
template <bool F16>
__device__ __forceinline__ bool any_not_finite(uint4 v) {
    constexpr uint32_t E = F16 ? 0x7C00u : 0x7F80u;
    bool bad = false;
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) bad |= (w[i] & E) == E || (w[i] & (E << 16)) == (E << 16);
    return bad;
}
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
// The larger of each half's values so far and those of eight more, signs aside: infinities and NaNs are the largest.
template <bool F16>
__device__ __forceinline__ u16x2 largest_exponents(u16x2 most, uint4 v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) most = __builtin_elementwise_max(most, __builtin_bit_cast(u16x2, w[i] & 0x7fff7fffu));
    return most;
}
template <bool F16>
__device__ __forceinline__ uint4 finite_part(uint4 v) {
    s16x8 b = __builtin_bit_cast(s16x8, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) b[e] = not_finite<F16>((uint16_t)b[e]) ? (short)0 : b[e];
    return __builtin_bit_cast(uint4, b);
}

// Infinities and NaNs among the values that a lane's row has seen: bit i of word i / 32 for its i-th
// output, in the order of its accumulators (an output per four consecutive d each).
template <int WORDS>
struct Special {
    uint32_t pos[WORDS], neg[WORDS];
    __device__ __forceinline__ bool any() const {
        uint32_t x = 0;
#pragma unroll
        for (int i = 0; i < WORDS; ++i) x |= pos[i] | neg[i];
        return x != 0;
    }
    // Calls add(i, infinity or NaN) for every output i that has seen one.
    template <typename F>
    __device__ __forceinline__ void apply(F add) const {
#pragma unroll 1
        for (int i = 0; i < 32 * WORDS; ++i) {
            uint32_t p = 0, n = 0;
#pragma unroll
            for (int k = 0; k < WORDS; ++k)
                if (k == i / 32) p = pos[k] >> (i % 32) & 1, n = neg[k] >> (i % 32) & 1;
            if (p | n) add(i, p & n ? __builtin_nanf("") : p ? INFINITY : -INFINITY);
        }
    }
    // The four outputs from number 4 j on, for which the key's values are v.
    template <bool F16>
    __device__ __forceinline__ void add(int j, uint2 v) {
        uint32_t p = 0, n = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint16_t b = (uint16_t)((e < 2 ? v.x : v.y) >> (16 * (e & 1)));
            const bool bad = not_finite<F16>(b), nan = bad && (b & (F16 ? 0x3FF : 0x7F));
            p |= (uint32_t)(bad && (nan || !(b & 0x8000))) << e;
            n |= (uint32_t)(bad && (nan || (b & 0x8000))) << e;
        }
        p <<= (4 * j) % 32;
        n <<= (4 * j) % 32;
#pragma unroll
        for (int i = 0; i < WORDS; ++i)
            if (i == 4 * j / 32) pos[i] |= p, neg[i] |= n;
    }
};

// What the kernels need beside the arguments, worked out on the host.
struct Plan {
    float c;          // |scale| log2 e, at least 1e-37 (so that -inf times it stays -inf)
    uint32_t flip;    // sign bits of a pair of 16-bit values where scale < 0: applied to q
    uint32_t magic;   // n / page = (n * magic) >> shift for 0 <= n < 2^31
    int shift;
    int G;            // query heads per key/value head
    int splits;       // parts that a row tile's keys are divided into, over workgroups
    int rows_lo, rows_hi;  // this launch takes the requests with rows_lo < rows <= rows_hi
    int64_t tiles;         // row tiles in the grid, per key/value head
    int each;              // many rows: row tiles of every request; 0: as many as it has tokens for
    int zero_rest;         // this launch writes the tokens that belong to no request (workgroups past `splits` only those)
};

__device__ __forceinline__ int page_of(const Plan& p, int key) {
    return (int)(((uint64_t)(uint32_t)key * p.magic) >> p.shift);
}

// Many rows: row tile `tile` of `bm` rows -> its request and its number in it: request r's tiles start at
// floor(cu[r] G / bm) + r, which leaves room for ceil(n_r G / bm), or at `each` r.  Returns false where there is none.
__device__ __forceinline__ bool find_tile(const AttentionArgs& a, const Plan& pl, int64_t tile, int bm, int& r, int& first) {
    const int G = pl.G;
    if (pl.each) {
        r = (uint32_t)tile / (uint32_t)pl.each;
        first = ((uint32_t)tile % (uint32_t)pl.each) * bm;
        return true;
    }
    int lo = 0;  // the last request whose tiles start at or before `tile`, by 64 probes at a time
    for (int n = a.R; n > 1;) {
        const int step = (n + 63) / 64, lane = threadIdx.x & 63, at = lo + lane * step;
        const bool before = lane * step < n && (int64_t)a.cu[at] * G / bm + at <= tile;
        const int k = __builtin_amdgcn_readfirstlane(__popcll(__ballot(before)));  // (the first is, the others in order)
        lo += (k > 0 ? k - 1 : 0) * step;
        n = min(step, a.R - lo);
    }
    r = lo;
    first = (int)(tile - ((int64_t)a.cu[lo] * G / bm + lo)) * bm;
    return first >= 0;
}

// The first key that a token at position pos sees.  A token before position 0 (fewer cached tokens than new ones) counts
// as at 0, where the answer is 0 too: its own position minus a window of up to 2^31 - 1 would not fit into 32 bits.
__device__ __forceinline__ int first_seen(const AttentionArgs& a, int pos) {
    return a.window ? max(0, max(pos, 0) - a.window + 1) : 0;
}

// One request's rows and keys, as a tile sees them.
struct Rows {
    int n, kv, pos0;  // new tokens (at most max_q), keys, position of token 0
    int t0;           // its packed index
    int key_begin, key_end;
};
__device__ __forceinline__ Rows rows_of(const AttentionArgs& a, int r, int first_row, int bm, int G) {
    Rows w;
    w.t0 = min(max(a.cu[r], 0), a.T);
    const int all = min(max(a.cu[r + 1], w.t0), a.T) - w.t0;
    const int64_t room = (int64_t)a.max_pages * a.page;
    const int kv = a.kv_len[r] < 0 ? 0 : a.kv_len[r];
    w.kv = kv < room ? kv : (int)room;
    w.pos0 = w.kv - all;
    w.n = all < a.max_q ? all : a.max_q;
    const int last = min(w.n * G, first_row + bm) - 1;
    w.key_end = w.kv;
    w.key_begin = first_seen(a, w.pos0 + first_row / G);
    if (a.causal) w.key_end = min(w.kv, w.pos0 + last / G + 1);
    return w;
}

// Tokens that belong to no request (before the first one's, behind the last one's) get zeros: their rows (token and
// head) go to the grid's workgroups in turn, a piece of 16 bytes per thread.  A step padded to a fixed number of tokens
// has many of them: a call with 8,192 tokens of which two requests have 2 (32 heads over 8, D = 128, 67 MB of zeros)
// takes 16 us, without them 13; by one workgroup per key/value head, a token after the other, 1,174.
template <int DP>
__device__ __forceinline__ void zero_rest(const AttentionArgs& a) {
    constexpr int LANES = DP <= 64 ? 8 : DP <= 128 ? 16 : 32;  // a row's
    const int begin = min(max(a.cu[0], 0), a.T), end = min(max(a.cu[a.R], begin), a.T);  // (no request: equal)
    const int64_t rows = (int64_t)(begin + a.T - end) * a.H;                               // (below 2^31)
    if (rows == 0) return;
    const int64_t wg = blockIdx.x + gridDim.x * (blockIdx.y + (int64_t)gridDim.y * blockIdx.z);
    const int64_t wgs = (int64_t)gridDim.x * gridDim.y * gridDim.z;
    const int share = blockDim.x / LANES, d = threadIdx.x % LANES * 8;
    for (int64_t i = wg * share + threadIdx.x / LANES; i < rows; i += wgs * share) {
        const int nth = (uint32_t)i / (uint32_t)a.H, h = (uint32_t)i % (uint32_t)a.H, t = nth < begin ? nth : nth - begin + end;
        if (d < a.D) *reinterpret_cast<uint4*>(a.out + t * a.o_tok + h * a.o_head + d) = make_uint4(0, 0, 0, 0);
        if (a.lse && d == 0) a.lse[(int64_t)t * a.H + h] = -INFINITY;
    }
}

// The larger of a lane's value and that of lane l XOR 32.
__device__ __forceinline__ float max_of_halves(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// What a lane of few_rows_kernel takes of a key's row.  The order of the dimensions inside a contraction is free: each lane
// loads PIECE neighbouring ones at a time (16 bytes where the row's width allows), which feed STEPS steps of 32.
template <int KIND, int DP>
struct Lanes {
    static_assert(KIND == CACHE_16 || DP % 64 == 0, "");  // (see few_dim)
    static constexpr int PIECE = KIND == CACHE_16 ? 8 : KIND == MXFP8 || DP % 128 != 0 ? 16 : 32;
    static constexpr int STEPS = PIECE / 8, PIECES = DP / 4 / PIECE;
    static constexpr int WORDS = KIND == MXFP8 ? 2 : 1;  // of codes, for eight values
    // The first of the eight dimensions of step ks that the lanes of `quad` hold.
    static __device__ __forceinline__ int dim(int ks, int quad) {
        return 32 * STEPS * (ks / STEPS) + PIECE * quad + 8 * (ks % STEPS);
    }
};
// A lane's share of a row, as loaded, and the 16-bit values of its steps.
template <int KIND, bool F16, int DP>
struct Share {
    typedef Lanes<KIND, DP> L;
    uint32_t w[L::PIECES * L::STEPS * L::WORDS];
    uint32_t scale[L::PIECES];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < L::PIECES * L::STEPS * L::WORDS; ++i) w[i] = 0;
#pragma unroll
        for (int i = 0; i < L::PIECES; ++i) scale[i] = 0;
    }
    // row + at, scales + scale_at: of this key and head; D: the row's length
    __device__ __forceinline__ void load(const uint8_t* row, uint32_t at, const uint8_t* scales, uint32_t scale_at, int quad, int D) {
        constexpr int N = L::STEPS * L::WORDS;  // words a piece
        typedef uint32_t words __attribute__((ext_vector_type(N)));
#pragma unroll
        for (int j = 0; j < L::PIECES; ++j) {
            const int d = 4 * L::PIECE * j + L::PIECE * quad;
            if (D != DP && d >= D) continue;
            const words v = *reinterpret_cast<const words*>(row + (at + (KIND == MXFP4 ? d / 2 : d)));
#pragma unroll
            for (int i = 0; i < N; ++i) w[N * j + i] = v[i];
            scale[j] = scales[scale_at + d / MX_BLOCK];
        }
    }
    __device__ __forceinline__ uint4 step(int ks) const {
        const float s = mx_scale_operand(scale[ks / L::STEPS]);
        if constexpr (KIND == MXFP4) return mx_decode16<KIND, F16>(make_uint2(w[ks], 0), s);
        else return mx_decode16<KIND, F16>(make_uint2(w[2 * ks], w[2 * ks + 1]), s);
    }
};
template <bool F16, int DP>
struct Share<CACHE_16, F16, DP> {
    uint4 v[DP / 32];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int ks = 0; ks < DP / 32; ++ks) v[ks] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ uint4 step(int ks) const { return v[ks]; }
};

// The four values from dimension d (a multiple of 4) on of a value's row: page `page`, place `at` in it.
template <int KIND, bool F16>
__device__ __forceinline__ uint2 four_of_value(const AttentionArgs& a, int kvh, int page, int at, int d) {
    const int64_t to = page * a.c_page + kvh * a.c_head + (int64_t)at * a.c_row;
    if constexpr (KIND == CACHE_16) {
        return *reinterpret_cast<const uint2*>(a.vc + to + d);
    } else {
        const uint8_t* row = reinterpret_cast<const uint8_t*>(a.vc) + to;
        const uint8_t byte = a.vs[page * a.s_page + kvh * a.s_head + (int64_t)at * a.s_row + d / MX_BLOCK];
        const uint32_t w = KIND == MXFP4 ? *reinterpret_cast<const uint16_t*>(row + d / 2) : *reinterpret_cast<const uint32_t*>(row + d);
        const uint4 v = mx_decode16<KIND, F16>(make_uint2(w, 0), mx_scale_operand(byte));
        return make_uint2(v.x, v.y);
    }
}

// ---------------------------------------------------------------------------------------------
// Few rows (generation): a workgroup takes a request's rows (at most 16) and one part of the keys; its four (or eight,
// see divide) waves take tiles of 32 keys in turn, each with its own running maximum, and join at the end.  Bound by
// reading K and V: both go from memory to registers in pieces of 16 bytes a lane, the next tile's while this one is
// worked on; V passes through the wave's own LDS to be transposed, so the waves never wait for each other.  64 requests
// of up to 8,192 keys (32 heads over 8, D = 128): 323 us, 5.3 TB/s (a copy of 2 GiB reaches 4.9).  One request of some
// 400 keys: 7.2 us, of which three loads that wait for each other (lengths, table, keys) take the most, and 4.0 for the
// join.  D = 256 (one wave per SIMD): the same 64 requests 646 us, 5.3 TB/s.  Four waves a workgroup | eight, us: one
// request of 100 keys 6.5 | 6.6, at D = 256 8.7 | 11.4, the 64 requests at D = 256 646 | 757 (eight spill), at D = 128
// and 64 the same.
//
// Microscaled blocks (KIND): a lane's pieces are smaller, so that more of the time is the chain of a tile's steps, and waves
// beside each other hide it: three per SIMD up to 128 dimensions (four up to 64), two above.  The same 64 requests, us, MXFP8 |
// MXFP4: 175 | 104 back to back (256 dimensions 349 | 186).  In short runs, whose clock is lower, 204 | 118 (256 dimensions 403 |
// 211, without that bound on registers 458 | 311); two tiles on their way in place of one, with fewer waves: 234 | 130.
template <int KIND, int DP, bool PAGE16>
constexpr int few_waves_per_simd() { return KIND == CACHE_16 ? 1 : (DP <= 64 ? 4 : DP <= 128 ? 3 : 2) - (PAGE16 ? 0 : 1); }

// W waves: 4, or 8 where the keys are not divided over workgroups.
template <int KIND, bool F16, int DP, bool PAGE16, int W>
__global__ __launch_bounds__(64 * W, (W == 8 ? 2 : few_waves_per_simd<KIND, DP, PAGE16>())) void few_rows_kernel(AttentionArgs a, Plan pl) {
    typedef Lanes<KIND, DP> L;
    constexpr int BM = FEW, BN = 32, KS = DP / 32, DT = DP / 16;
    // Rows of V 16 banks apart (mod 64); of microscaled blocks an odd multiple of 8, with which 8 rows written at one
    // dimension miss each other too: a fourth of the cycles that LDS loses to them otherwise.
    constexpr int VS = KIND != CACHE_16 ? DP + 16 : DP + ((DP / 2) % 64 == 16 || (DP / 2) % 64 == 48 ? 0 : 32);
    constexpr int OS = DP + 4;
    constexpr int WAVE_BYTES = BN * VS * 2 > BM * OS * 4 ? BN * VS * 2 : BM * OS * 4;
    __shared__ __align__(16) uint8_t lds[W * WAVE_BYTES];
    __shared__ float wave_m[W][BM], wave_l[W][BM];
    const int tid = threadIdx.x, lane = tid & 63, col = lane & 15, quad = lane >> 4;
    const int wave = PAGE16 ? __builtin_amdgcn_readfirstlane(tid >> 6) : tid >> 6;
    const int G = pl.G, kvh = blockIdx.x, r = blockIdx.y, split = blockIdx.z;
    if (pl.zero_rest) zero_rest<DP>(a);
    if (a.R == 0 || split >= pl.splits) return;
    const Rows w = rows_of(a, r, 0, BM, G);
    const int rows = w.n * G;
    if (rows <= pl.rows_lo || rows > pl.rows_hi) return;

    uint16_t* vl = reinterpret_cast<uint16_t*>(lds + wave * WAVE_BYTES);
    const int row = col, tok = row / G, pos = w.pos0 + tok;
    const bool live = row < rows;
    // the keys this lane's row sees: [see_lo, see_hi)
    const int see_hi = !live ? 0 : a.causal ? min(w.kv, pos + 1) : w.kv;
    const int see_lo = first_seen(a, pos);
    const int same_hi = a.causal ? min(w.kv, w.pos0 + 1) : w.kv;  // every live row sees keys in
    const int same_lo = first_seen(a, w.pos0 + (rows - 1) / G);          // [same_lo, same_hi)

    int64_t q_at = (int64_t)(w.t0 + tok) * a.q_tok + (int64_t)(kvh * G + row - tok * G) * a.q_head + L::PIECE * quad;
    asm volatile("" : "+v"(q_at));  // worked out once, and not in front of every load
    s16x8 q[KS];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (live && L::dim(ks, quad) < a.D) {
            v = *reinterpret_cast<const uint4*>(a.q + q_at + L::dim(ks, 0));
            v.x ^= pl.flip; v.y ^= pl.flip; v.z ^= pl.flip; v.w ^= pl.flip;
        }
        q[ks] = __builtin_bit_cast(s16x8, v);
    }

    // this part's tiles of 32 keys
    const int t_begin = w.key_begin / BN, t_end = (w.key_end + BN - 1) / BN;
    const int per = max(0, (t_end - t_begin + pl.splits - 1) / pl.splits);
    const int t0 = t_begin + split * per, t1 = min(t_end, t0 + per);
    const int32_t* table = a.table + r * a.table_stride;

    const uint32_t col_at = PAGE16 ? col * (uint32_t)a.c_row : 0, col_scale = PAGE16 ? col * (uint32_t)a.s_row : 0;
    int page_id[2];
    auto fetch_ids = [&](int t) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if constexpr (PAGE16) {  // the 16 keys are in one page
                const int key = t * BN + 16 * h;
                page_id[h] = -1;
                if (t < t1 && key + 16 > w.key_begin && key < w.key_end) page_id[h] = table[page_of(pl, key)];
                continue;
            }
            const int key = t * BN + 16 * h + col;
            page_id[h] = -1;
            if (t < t1 && key >= w.key_begin && key < w.key_end) page_id[h] = table[page_of(pl, key)];
        }
    };
    Share<KIND, F16, DP> kr[2], vr[2];
    int ok_next[2];
    auto fetch_kv = [&](int t) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int key = t * BN + 16 * h + col;
            kr[h].clear();
            vr[h].clear();
            if constexpr (PAGE16) {
                const int id = __builtin_amdgcn_readfirstlane(page_id[h]), first = t * BN + 16 * h, in_page = first - page_of(pl, first) * a.page;
                ok_next[h] = id >= 0 && id < a.n_pages && key >= w.key_begin && key < w.key_end;
                if (!ok_next[h]) continue;
                const int64_t at = id * a.c_page + kvh * a.c_head + in_page * a.c_row;
                const int64_t sat = id * a.s_page + kvh * a.s_head + in_page * a.s_row;
                kr[h].load(reinterpret_cast<const uint8_t*>(a.kc) + at, col_at, a.ks + sat, col_scale, quad, a.D);
                vr[h].load(reinterpret_cast<const uint8_t*>(a.vc) + at, col_at, a.vs + sat, col_scale, quad, a.D);
                continue;
            }
            ok_next[h] = page_id[h] >= 0 && page_id[h] < a.n_pages;
            if constexpr (KIND == CACHE_16) {
                const int64_t at = page_id[h] * a.c_page + kvh * a.c_head + (int64_t)(key - page_of(pl, key) * a.page) * a.c_row + 8 * quad;
                if (!ok_next[h]) continue;
                if (a.D == DP) {
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) kr[h].v[ks] = *reinterpret_cast<const uint4*>(a.kc + at + 32 * ks);
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) vr[h].v[ks] = *reinterpret_cast<const uint4*>(a.vc + at + 32 * ks);
                } else {
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks)
                        if (32 * ks + 8 * quad < a.D) {
                            kr[h].v[ks] = *reinterpret_cast<const uint4*>(a.kc + at + 32 * ks);
                            vr[h].v[ks] = *reinterpret_cast<const uint4*>(a.vc + at + 32 * ks);
                        }
                }
            } else {
                if (!ok_next[h]) continue;
                int me = lane;
                if constexpr (W == 8 && DP > 192) asm volatile("" : "+v"(me));  // (no register to keep what follows from it)
                const int in_page = key - page_of(pl, key) * a.page;
                const int64_t at = page_id[h] * a.c_page + kvh * a.c_head + (int64_t)in_page * a.c_row;
                const int64_t sat = page_id[h] * a.s_page + kvh * a.s_head + (int64_t)in_page * a.s_row;
                kr[h].load(reinterpret_cast<const uint8_t*>(a.kc) + at, 0, a.ks + sat, 0, me >> 4, a.D);
                vr[h].load(reinterpret_cast<const uint8_t*>(a.vc) + at, 0, a.vs + sat, 0, me >> 4, a.D);
            }
        }
    };

    f32x4 o[DT];
#pragma unroll
    for (int d = 0; d < DT; ++d) o[d] = f32x4{0, 0, 0, 0};
    float m = -INFINITY, l = 0.0f;
    Special<(4 * DT + 31) / 32> seen = {};

    int t = t0 + wave;
    fetch_ids(t);
    fetch_kv(t);
    fetch_ids(t + W);
    for (; t < t1; t += W) {
        f32x4 s[2];
        const bool mixed = t * BN < same_lo || (t + 1) * BN > same_hi;
        uint64_t there[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            s[h] = f32x4{0, 0, 0, 0};
            there[h] = __ballot(ok_next[h]);
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                s[h] = mfma16<F16>(__builtin_bit_cast(s16x8, kr[h].step(ks)), q[ks], s[h]);
                *reinterpret_cast<uint4*>(vl + (16 * h + col) * VS + L::dim(ks, quad)) = vr[h].step(ks);
            }
        }
        bool special = false;
        if (mixed) {
            u16x2 most = {0, 0};
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) most = largest_exponents<F16>(most, vr[h].step(ks));
            special = __any(not_finite<F16>(most.x) || not_finite<F16>(most.y));
            if (special)
#pragma unroll 1
                for (int i = 0; i < 2 * KS; ++i) {  // the pieces this lane has stored
                    uint4* at = reinterpret_cast<uint4*>(vl + (16 * (i / KS) + col) * VS + L::dim(i % KS, quad));
                    *at = finite_part<F16>(*at);
                }
        }
        fetch_kv(t + W);
        fetch_ids(t + 2 * W);
        // masks, running maximum
        float top = -INFINITY;
        const bool all_there = (there[0] & there[1] & 0xffff) == 0xffff;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (mixed || !all_there) {
                    const int k = 4 * quad + e, key = t * BN + 16 * h + k;
                    if (key < see_lo || key >= see_hi || !((there[h] >> k) & 1)) s[h][e] = -INFINITY;
                }
                top = fmaxf(top, s[h][e]);
            }
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        const float m_new = fmaxf(m, top);
        const float mc = m_new == -INFINITY ? 0.0f : m_new * pl.c;
        if (__any(m_new > m)) {
            const float keep = __builtin_amdgcn_exp2f(__builtin_fmaf(m, pl.c, -mc));
            l *= keep;
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[d][e] *= keep;
            m = m_new;
        }
        float p[8];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                p[4 * h + e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[h][e], pl.c, -mc));
                l += p[4 * h + e];
            }
        const s16x8 pb = pack8<F16>(p);
        // O^T += V^T P^T: keys in the order 16 h + 4 quad + e
        const uint16_t* va = vl + (4 * quad + (col >> 2)) * VS + 4 * (col & 3);
#pragma unroll
        for (int d = 0; d < DT; ++d) {
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(va + 16 * d));
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(va + 16 * VS + 16 * d));
            o[d] = mfma16<F16>(__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7), pb, o[d]);
        }
        if (special) {
#pragma unroll 1
            for (int key = max(t * BN, w.key_begin); key < min((t + 1) * BN, w.key_end); ++key) {
                const int id = table[page_of(pl, key)];
                if (id < 0 || id >= a.n_pages) continue;
                if (key >= see_lo && key < see_hi)  // (also where its weight is 0)
#pragma unroll 1
                    for (int d = 0; d < DT; ++d)
                        if (16 * d + 4 * quad < a.D) seen.template add<F16>(d, four_of_value<KIND, F16>(a, kvh, id, key - page_of(pl, key) * a.page, 16 * d + 4 * quad));
            }
        }
    }
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);

    // join the waves
    float* ol = reinterpret_cast<float*>(lds + wave * WAVE_BYTES);
    __syncthreads();
    if (quad == 0) {
        wave_m[wave][col] = m;
        wave_l[wave][col] = l;
    }
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) ol[col * OS + 16 * d + 4 * quad + e] = o[d][e];
    if (seen.any()) seen.apply([&](int i, float x) { ol[col * OS + 4 * (i & ~3) + 4 * quad + (i & 3)] += x; });
    __syncthreads();
    const int live_rows = rows;
    const int64_t part = ((int64_t)r * a.Hkv + kvh) * pl.splits + split;
    for (int i = tid; i < live_rows * (DP / 4); i += 64 * W) {
        const int c = i / (DP / 4), d = i % (DP / 4) * 4;
        float M = -INFINITY;
#pragma unroll
        for (int x = 0; x < W; ++x) M = fmaxf(M, wave_m[x][c]);
        const float Mc = M == -INFINITY ? 0.0f : M * pl.c;
        float L = 0.0f;
        f32x4 acc = {0, 0, 0, 0};
#pragma unroll
        for (int x = 0; x < W; ++x) {
            const float f = __builtin_amdgcn_exp2f(__builtin_fmaf(wave_m[x][c], pl.c, -Mc));  // 0: it saw no key of the row
            L = __builtin_fmaf(f, wave_l[x][c], L);
            const f32x4 v = *reinterpret_cast<const f32x4*>(lds + x * WAVE_BYTES + (c * OS + d) * 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[e] = __builtin_fmaf(f, v[e], acc[e]);
        }
        if (pl.splits > 1) {
            float* wp = a.ws + part * (BM * (DP + 2));
            *reinterpret_cast<f32x4*>(wp + c * DP + d) = acc;
            if (d == 0) {
                wp[BM * DP + 2 * c] = M * pl.c;
                wp[BM * DP + 2 * c + 1] = L;
            }
        } else {
            const int rw = c;
            const int64_t tk = w.t0 + rw / G;
            const int head = kvh * G + rw % G;
            const bool none = L == 0.0f;
            if (d < a.D) {
                uint16_t b[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) b[e] = from_f32<F16>(none ? 0.0f : acc[e] / L);
                uint2 st = make_uint2(b[0] | (uint32_t)b[1] << 16, b[2] | (uint32_t)b[3] << 16);
                *reinterpret_cast<uint2*>(a.out + tk * a.o_tok + (int64_t)head * a.o_head + d) = st;
            }
            if (a.lse && d == 0) a.lse[tk * a.H + head] = none ? -INFINITY : (M * pl.c + __log2f(L)) * LN2;
        }
    }
}

// Place of the 16-byte piece `piece` in row `row` of a tile [keys][DP] in LDS.  Three accesses have to
// miss each other's banks (64 of 4 bytes): 16 rows at one piece (K's operand), 4 neighbouring rows at 4
// pieces (V's transposing read), and the same 4 x 4 as the staging writes it.
template <int DP>
__device__ __forceinline__ int turn(int row) {
    if constexpr (DP % 128 == 0) return 4 * (row & 3) + ((row >> 2) & 3);
    if constexpr (DP % 128 == 64) return 4 * ((row >> 1) & 1) + ((row >> 2) & 3);
    return (row >> 2) & 3;
}
template <int DP>
__device__ __forceinline__ int place(int row, int piece) {
    return piece ^ turn<DP>(row);
}
// Address in LDS of piece `piece` (a constant) moved by a lane's own share of it: `lane_at` holds the
// tile, the row and 16 (own ^ turn), own and piece having no bits in common; the turn stays within
// BLOCK bytes, to a multiple of which tile and rows are aligned.
template <int DP>
__device__ __forceinline__ uint32_t piece_at(uint32_t lane_at, int piece) {
    constexpr int BLOCK = DP % 128 == 0 ? 256 : DP % 128 == 64 ? 128 : 64;
    return (lane_at ^ (uint32_t)(16 * piece & (BLOCK - 1))) + (uint32_t)(16 * piece & ~(BLOCK - 1));
}
__device__ __forceinline__ uint32_t lds_offset(const void* p) {
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p;
}
typedef const __attribute__((address_space(3))) s16x8* lds_s16x8;

__device__ const uint4 zeros[1] = {};  // what a lane reads for a key or a dimension that is not there

// ---------------------------------------------------------------------------------------------
// Many rows (prompts): a workgroup takes 256 rows, 32 per wave (two waves per SIMD); tiles of BN keys and values go from
// memory straight into LDS for all eight waves, three tiles ahead, one barrier a tile.  Where the rows of the next 512
// keys lie is looked up at a time, a key per thread.  64 keys a tile up to 128 dimensions, 32 above, where four tiles of
// 64 would not fit into LDS (32 at D = 128: 1290 us in place of 784 at the time).
//
// Bound by the vector instructions of the softmax beside the matrix instructions: per 256 x 64 scores a SIMD has 64
// products of 32 cycles and some 390 vector instructions of 4 to 8, which overlap only in part.  2 requests of up to
// 2,048 tokens against 16,384 keys (32 heads over 8, D = 128): 672 to 760 us by the card and its clock, 790 to 890
// TFLOP/s; 32 requests of 256 tokens (8 heads over 2, D = 256): 44 us.  LDS is busy 19 % of the time, without conflicts.  Measured and not kept: 64 rows a wave with one
// wave per SIMD and the next scores between the exponentials (792 us); 128 rows a workgroup (766); two groups of waves
// in turns (712 to 740).
//
// Microscaled blocks (KIND): codes do not go straight into LDS, which holds 16-bit values: a thread loads those of the tile
// after next, converts what it has of the next one, and writes them where the loads above would (two tiles in LDS).  The
// same 2 requests, us, MXFP8 | MXFP4 | 16-bit values, back to back on one card: 758 | 747 | 686 (D = 64, four waves a SIMD: 466 |
// 460 | 407; with two 531 | 550).  The 32 requests at D = 256: 46 | 44 | 43, of 8 tiles at most a workgroup, one after the
// other.
template <int KIND, bool F16, int DP, int BN>
__global__ __launch_bounds__(2 * MANY, (KIND != CACHE_16 && DP <= 64 ? 4 : 2)) void many_rows_kernel(AttentionArgs a, Plan pl) {
    constexpr int BM = MANY, KS = DP / 16, DT = DP / 32, KT = BN / 32;
    // no registers to spare: what can be is worked out anew where it is needed
    constexpr bool TIGHT = KIND != CACHE_16 && (DP > 192 || DP <= 64);
    constexpr int RUNS = BN * DP / 8 / 64, WAVES = MANY / 32;  // loads of 64 16-byte pieces a tile of K or V takes
    constexpr int PIECES = (RUNS + WAVES - 1) / WAVES;         // of them, per wave
    constexpr int STAGES = KIND == CACHE_16 ? 4 : 2;           // tiles in LDS
    constexpr int BLOCK = 2 * MANY;                            // keys looked up at a time, one per thread
    __shared__ __align__(256) uint16_t ktile[STAGES][BN * DP];
    __shared__ __align__(256) uint16_t vtile[STAGES][BN * DP];
    __shared__ int64_t row_at[2][BLOCK];             // of block b, in [b % 2]: offset of each key's row, -1: none
    __shared__ int64_t scales_at[KIND == CACHE_16 ? 1 : 2][KIND == CACHE_16 ? 1 : BLOCK];  // and of its scales
    __shared__ uint64_t missing_at[2][BLOCK / 64];  // keys in range whose page is not in the pool
    __shared__ int bad_at[4];                       // V of tile t, in [t % 4], holds what is not finite
    __shared__ Special<(16 * DT + 31) / 32> seen_at[2 * MANY];  // (in LDS: it is hardly ever used)
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), col = lane & 31, half = lane >> 5;
    const int G = a.H / a.Hkv;
    const int kvh = blockIdx.x % a.Hkv;
    const int64_t tile = pl.tiles - 1 - blockIdx.x / a.Hkv;  // the longest rows first
    const int split = blockIdx.y;
    if (pl.zero_rest) zero_rest<DP>(a);
    if (a.R == 0 || split >= pl.splits) return;
    int r, first;
    if (!find_tile(a, pl, tile, BM, r, first)) return;
    const Rows w = rows_of(a, r, first, BM, G);
    const int rows = w.n * G;
    if (first >= rows || rows <= pl.rows_lo || rows > pl.rows_hi) return;

    const int row = first + 32 * wave + col, tok = row / G, pos = w.pos0 + tok;
    const bool live = row < rows;
    const int see_hi = !live ? 0 : a.causal ? min(w.kv, pos + 1) : w.kv;
    const int see_lo = first_seen(a, pos);
    // keys that every row of the workgroup sees, and that every (any) row of the wave sees
    const int last = min(rows, first + BM) - 1;
    const int same_hi = a.causal ? min(w.kv, w.pos0 + first / G + 1) : w.kv;
    const int same_lo = first_seen(a, w.pos0 + last / G);
    const int wfirst = first + 32 * wave, wlast = min(rows - 1, wfirst + 31);
    const int wave_hi = wfirst >= rows ? 0 : a.causal ? min(w.kv, w.pos0 + wlast / G + 1) : w.kv;
    const int wave_lo = first_seen(a, w.pos0 + wfirst / G);
    const int wsame_hi = a.causal ? min(w.kv, w.pos0 + wfirst / G + 1) : w.kv;
    const int wsame_lo = first_seen(a, w.pos0 + wlast / G);

    const int head = kvh * G + row - tok * G;
    int64_t q_at = (int64_t)(w.t0 + tok) * a.q_tok + (int64_t)head * a.q_head + 8 * half;
    asm volatile("" : "+v"(q_at));  // worked out once, and not in front of every load
    s16x8 q[KS];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (live && 16 * ks + 8 * half < a.D) {
            v = *reinterpret_cast<const uint4*>(a.q + q_at + 16 * ks);
            v.x ^= pl.flip; v.y ^= pl.flip; v.z ^= pl.flip; v.w ^= pl.flip;
        }
        q[ks] = __builtin_bit_cast(s16x8, v);
    }

    const int t_begin = w.key_begin / BN, t_end = (w.key_end + BN - 1) / BN;
    const int per = max(0, (t_end - t_begin + pl.splits - 1) / pl.splits);
    const int t0 = t_begin + split * per, t1 = min(t_end, t0 + per);
    const int32_t* table = a.table + r * a.table_stride;

    // Where the rows of a block of keys lie, a thread per key: find() starts the table's load, note() ends it.  A key that
    // is not this part's has the page INT32_MIN, which no entry of the table may be taken for.
    auto find = [&](int b) {
        const int key = b * BLOCK + tid;
        return key >= t0 * BN && key < t1 * BN && key >= w.key_begin && key < w.key_end ? max(table[page_of(pl, key)], -1) : INT32_MIN;
    };
    auto note = [&](int b, int id) {
        const int key = b * BLOCK + tid;
        const bool ok = id >= 0 && id < a.n_pages;
        row_at[b & 1][tid] = ok ? id * a.c_page + (int64_t)(key - page_of(pl, key) * a.page) * a.c_row : -1;
        if constexpr (KIND != CACHE_16)
            scales_at[b & 1][tid] = id * a.s_page + (int64_t)(key - page_of(pl, key) * a.page) * a.s_row;
        const uint64_t missing = __ballot(!ok && id != INT32_MIN);
        if (lane == 0) missing_at[b & 1][wave] = missing;
    };
    const uint16_t* kbase = a.kc + kvh * a.c_head;
    const uint16_t* vbase = a.vc + kvh * a.c_head;
    auto fetch = [&](int t) {
        int me = lane;
        if constexpr (DP > 128) asm volatile("" : "+v"(me));  // worked out anew each time: there are no registers to keep it
        const int64_t* rows_at = &row_at[t * BN / BLOCK & 1][t * BN % BLOCK];
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const int run = wave + WAVES * i, at = 64 * run + me;
            if (RUNS % WAVES && run >= RUNS) break;
            const int row = at / (DP / 8), d = 8 * place<DP>(row, at % (DP / 8));
            const int64_t from = rows_at[row];
            const bool none = from < 0 || d >= a.D;
            load_to_lds(none ? (const uint16_t*)zeros : kbase + from + d, &ktile[t % STAGES][run * 512]);
            load_to_lds(none ? (const uint16_t*)zeros : vbase + from + d, &vtile[t % STAGES][run * 512]);
        }
    };

    // Microscaled blocks: a thread loads 16 values of a key at a time, a tile ahead, and puts them into LDS as 16-bit ones.
    constexpr int UNITS = BN * DP / 16, SHARES = (2 * UNITS + BLOCK - 1) / BLOCK;  // of K, and as many of V; a thread's
    uint4 raw[SHARES];
    uint32_t raw_scale[SHARES];
    auto ask = [&](int t) {
        int me = lane;
        if constexpr (DP > 128 || TIGHT) asm volatile("" : "+v"(me));  // (as in fetch)
        const int64_t* rows_at = &row_at[t * BN / BLOCK & 1][t * BN % BLOCK];
        const int64_t* srows_at = &scales_at[t * BN / BLOCK & 1][t * BN % BLOCK];
#pragma unroll
        for (int i = 0; i < SHARES; ++i) {
            const int u = BLOCK * i + 64 * wave;  // (UNITS is a multiple of 64: a wave's are all of K or all of V)
            raw[i] = make_uint4(0, 0, 0, 0);
            raw_scale[i] = 0;
            if (u >= 2 * UNITS) break;
            const bool of_v = u >= UNITS;
            const int at = u - (of_v ? UNITS : 0) + me, row = at / (DP / 16), d = at % (DP / 16) * 16;
            const int64_t from = rows_at[row];
            if (from < 0 || d >= a.D) continue;
            const uint8_t* codes = reinterpret_cast<const uint8_t*>(of_v ? a.vc : a.kc) + kvh * a.c_head + from;
            if constexpr (KIND == MXFP4) {
                const uint2 v = *reinterpret_cast<const uint2*>(codes + d / 2);
                raw[i].x = v.x;
                raw[i].y = v.y;
            } else {
                raw[i] = *reinterpret_cast<const uint4*>(codes + d);
            }
            raw_scale[i] = (of_v ? a.vs : a.ks)[kvh * a.s_head + srows_at[row] + d / MX_BLOCK];
        }
    };
    auto put = [&](int t) {
        int me = lane;
        if constexpr (DP > 128 || TIGHT) asm volatile("" : "+v"(me));
#pragma unroll
        for (int i = 0; i < SHARES; ++i) {
            const int u = BLOCK * i + 64 * wave;
            if (u >= 2 * UNITS) break;
            const bool of_v = u >= UNITS;
            const int at = u - (of_v ? UNITS : 0) + me, row = at / (DP / 16), piece = at % (DP / 16) * 2;
            uint16_t* to = (of_v ? vtile[t % STAGES] : ktile[t % STAGES]) + row * DP;
            const float s = mx_scale_operand(raw_scale[i]);
            const uint2 lo = make_uint2(raw[i].x, raw[i].y), hi = KIND == MXFP4 ? make_uint2(raw[i].y, 0) : make_uint2(raw[i].z, raw[i].w);
            *reinterpret_cast<uint4*>(to + 8 * place<DP>(row, piece)) = mx_decode16<KIND, F16>(lo, s);
            *reinterpret_cast<uint4*>(to + 8 * place<DP>(row, piece + 1)) = mx_decode16<KIND, F16>(hi, s);
        }
    };

    f32x16 o[DT];
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[d][e] = 0.0f;
    float m = -INFINITY, l = 0.0f;
    bool seen_yet = false;  // of the wave: its lanes' Special are in use

    // the lane's row of K and 16-byte piece of it; its key in a run of four of V, and its half of a piece
    const uint32_t k_lane = lds_offset(ktile) + 2 * DP * col + 16 * (half ^ turn<DP>(col));
    const int vkey = 4 * half + ((lane & 15) >> 2), vpiece = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
    const uint32_t v_lane = lds_offset(vtile) + 2 * DP * vkey + 16 * (vpiece ^ turn<DP>(vkey)) + 8 * (lane & 1);

    if (t0 < t1) {
        const int b = t0 * BN / BLOCK;
        const int id0 = find(b), id1 = find(b + 1);
        note(b, id0);
        note(b + 1, id1);
        if (tid < 4) bad_at[tid] = 0;
        __syncthreads();
        if constexpr (KIND == CACHE_16) {
            for (int t = t0; t < min(t0 + STAGES - 1, t1); ++t) fetch(t);
        } else {
            ask(t0);
            put(t0);
            if (t0 + 1 < t1) ask(t0 + 1);
        }
    }
    for (int t = t0; t < t1; ++t) {
        // the two tiles after this one may still be on their way
        if constexpr (KIND == CACHE_16) {
            if (t + STAGES - 2 < t1) loaded_to_lds<(STAGES - 2) * 2 * (RUNS / WAVES)>();
            else loaded_to_lds<0>();
        }
        __syncthreads();  // this tile is in LDS, the previous one has been read
        int id = INT32_MIN;
        const bool turn_over = t * BN % BLOCK == 0;  // the block before this one is done with
        if (turn_over) id = find(t * BN / BLOCK + 1);
        if constexpr (KIND == CACHE_16) {
            if (t + STAGES - 1 < t1) fetch(t + STAGES - 1);
        } else {
            if (t + 1 < t1) put(t + 1);
            if (t + 2 < t1) ask(t + 2);
        }
        if (tid == 0) bad_at[(t + 2) & 3] = 0;
        bool special = false;
        if (t * BN < same_lo || (t + 1) * BN > same_hi) {  // the rows' masks differ here
            int me = lane;
            if constexpr (TIGHT) asm volatile("" : "+v"(me));
#pragma unroll 1
            for (int i = 64 * wave + me; i < 64 * RUNS; i += 64 * WAVES) {
                uint16_t* at = &vtile[t % STAGES][8 * i];
                const uint4 v = *reinterpret_cast<const uint4*>(at);
                if (any_not_finite<F16>(v)) {
                    bad_at[t & 3] = 1;
                    *reinterpret_cast<uint4*>(at) = finite_part<F16>(v);
                }
            }
            __syncthreads();
            special = __builtin_amdgcn_readfirstlane(bad_at[t & 3]);
        }
        if (t * BN < wave_hi && (t + 1) * BN > wave_lo) {  // some row of this wave sees the tile
        uint32_t missing[KT];
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) missing[kt] = __builtin_amdgcn_readfirstlane(
                (uint32_t)(missing_at[t * BN / BLOCK & 1][t * BN % BLOCK / 64] >> (t * BN % 64 + 32 * kt)));
        f32x16 s[KT];
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
            for (int e = 0; e < 16; ++e) s[kt][e] = 0.0f;
        const uint32_t ka = k_lane + t % STAGES * (2 * BN * DP), va = v_lane + t % STAGES * (2 * BN * DP);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
                const uint32_t at = piece_at<DP>(ka, 2 * ks) + 64 * DP * kt;
                s[kt] = mfma32<F16>(*(lds_s16x8)at, q[ks], s[kt]);
            }
        // four operands ahead of their products (the compiler reads each just before it), two where registers are short
        constexpr int AHEAD = TIGHT && DP > 64 ? 2 : 4;
        __builtin_amdgcn_sched_group_barrier(0x100, AHEAD, 0);
#pragma unroll
        for (int x = 0; x < (KS * KT - AHEAD) / 2; ++x) {
            __builtin_amdgcn_sched_group_barrier(0x8, 2, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x8, AHEAD, 0);
        float top = -INFINITY;
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
            if (t * BN < wsame_lo || (t + 1) * BN > wsame_hi || missing[kt]) {
                // bit k: the row sees key k of these 32; the lane's are 8 (e / 4) + e % 4 after its first one
                const int at = t * BN + 32 * kt, lo = min(max(see_lo - at, 0), 32), hi = min(max(see_hi - at, 0), 32);
                const uint32_t sees = ((uint32_t)(((uint64_t)1 << hi) - 1) & ~(uint32_t)(((uint64_t)1 << lo) - 1) & ~missing[kt]) >> (4 * half);
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (!((sees >> (8 * (e >> 2) + (e & 3))) & 1)) s[kt][e] = -INFINITY;
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) top = fmaxf(top, s[kt][e]);
        }
        const float m_new = fmaxf(m, max_of_halves(top));
        if (__any((m_new - m) * pl.c > LAG)) {
            const float keep = m_new == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f((m - m_new) * pl.c);  // (before the first key: 0)
            l *= keep;
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int e = 0; e < 16; ++e) o[d][e] *= keep;
            m = m_new;
        }
        const float mc = m == -INFINITY ? 0.0f : m * pl.c;
        float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                s[kt][e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[kt][e], pl.c, -mc));
                sum[e & 3] += s[kt][e];
            }
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
#pragma unroll
        for (int ss = 0; ss < BN / 16; ++ss) {
            float p[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) p[e] = s[ss / 2][8 * (ss % 2) + e];
            const s16x8 pb = pack8<F16>(p);
#pragma unroll
            for (int d = 0; d < DT; ++d) {
                // keys 16 ss + vkey, and 8 further on, whose turn differs in one bit
                const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(piece_at<DP>(va, 4 * d) + 32 * DP * ss));
                const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (lds_s16x4)(piece_at<DP>(va, (4 * d) ^ 2) + 32 * DP * ss + 16 * DP));
                o[d] = mfma32<F16>(__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7), pb, o[d]);
            }
        }
        if (special) {
            Special<(16 * DT + 31) / 32> seen = {};
            if (seen_yet) seen = seen_at[tid];
            seen_yet = true;
#pragma unroll 1
            for (int key = max(t * BN, w.key_begin); key < min((t + 1) * BN, w.key_end); ++key) {
                const int page = table[page_of(pl, key)];
                if (page < 0 || page >= a.n_pages) continue;
                if (key >= see_lo && key < see_hi)  // (also where its weight is 0)
#pragma unroll 1
                    for (int j = 0; j < 4 * DT; ++j)  // accumulators 4 j .. of the lane: d = 8 j + 4 half ..
                        if (8 * j + 4 * half < a.D) seen.template add<F16>(j, four_of_value<KIND, F16>(a, kvh, page, key - page_of(pl, key) * a.page, 8 * j + 4 * half));
            }
            seen_at[tid] = seen;
        }
        }
        if (turn_over) note(t * BN / BLOCK + 1, id);
    }
    l += __shfl_xor(l, 32);
    // the lane's row once more: there are no registers to keep it through the tiles
    int me = lane;
    if constexpr (TIGHT) asm volatile("" : "+v"(me));
    const int end_col = me & 31, end_half = me >> 5, end_row = first + 32 * wave + end_col, end_tok = end_row / G;
    const bool end_live = end_row < rows;
    if (pl.splits > 1) {
        float* wp = a.ws + ((tile * a.Hkv + kvh) * pl.splits + split) * (BM * (DP + 2));
        const int c = 32 * wave + end_col;
        if (end_live) {
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int e = 0; e < 16; e += 4)
                    *reinterpret_cast<f32x4*>(wp + c * DP + 32 * d + 2 * e + 4 * end_half) =
                        f32x4{o[d][e], o[d][e + 1], o[d][e + 2], o[d][e + 3]};
            if (end_half == 0) {
                wp[BM * DP + 2 * c] = m * pl.c;
                wp[BM * DP + 2 * c + 1] = l;
            }
            if (seen_yet) seen_at[tid].apply([&](int i, float x) { wp[c * DP + 2 * (i & ~3) + 4 * end_half + (i & 3)] += x; });
        }
        return;
    }
    if (end_live) {
        const bool none = l == 0.0f;
        const float inv = none ? 0.0f : 1.0f / l;  // (o is 0 there)
        int64_t o_at = (int64_t)(w.t0 + end_tok) * a.o_tok + (int64_t)(kvh * G + end_row - end_tok * G) * a.o_head + 4 * end_half;
        asm volatile("" : "+v"(o_at));
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int e = 0; e < 16; e += 4)
                if (32 * d + 2 * e + 4 * end_half < a.D) {
                    uint32_t b[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x) b[x] = from_f32<F16>(o[d][e + x] * inv);
                    *reinterpret_cast<uint2*>(a.out + o_at + 32 * d + 2 * e) = make_uint2(b[0] | b[1] << 16, b[2] | b[3] << 16);
                }
        if (seen_yet)
            seen_at[tid].apply([&](int i, float x) {
                if (2 * (i & ~3) + 4 * end_half >= a.D) return;
                uint16_t* at = a.out + o_at + 2 * (i & ~3) + (i & 3);
                *at = from_f32<F16>(to_f32<F16>(*at) + x);
            });
        if (a.lse && end_half == 0) a.lse[(int64_t)(w.t0 + end_tok) * a.H + kvh * G + end_row - end_tok * G] = none ? -INFINITY : (m * pl.c + __log2f(l)) * LN2;
    }
}

// Joins the parts of a row tile: THREADS threads a row, each with four neighbouring d of every SUBS-th part, eight parts
// on their way at a time.  What it takes is the chain of loads, not their bytes: a token against 16,000 keys in 125 parts
// (8 heads over 2, D = 128) took 84 us with a wave a row and one part after the other, and takes 12.  A workgroup a row
// where the rows are few, a wave a row where a tile has 256 of them.
template <bool F16, int DP, int BM, int THREADS>
__global__ __launch_bounds__(256) void join_kernel(AttentionArgs a, Plan pl) {
    constexpr int SHARE = 256 / THREADS, PER = DP / 4, SUBS = THREADS / PER, PART = BM * (DP + 2), AHEAD = 8;
    __shared__ float factor[SHARE][256], most[4], total[4];
    __shared__ __align__(16) f32x4 sums[256];
    const int tid = threadIdx.x, wave = tid >> 6, own = tid % THREADS, mine = tid / THREADS;
    const int G = pl.G;
    const int64_t wg = blockIdx.x;
    const int c0 = (int)(wg % (BM / SHARE)) * SHARE, kvh = (int)(wg / (BM / SHARE) % a.Hkv);
    const int64_t tile = wg / (BM / SHARE) / a.Hkv;
    if (a.R == 0) return;
    int r, first;
    if (BM == FEW) {
        r = (int)tile;
        first = 0;
    } else if (!find_tile(a, pl, tile, BM, r, first)) {
        return;
    }
    const Rows w = rows_of(a, r, first, BM, G);
    const int rows = w.n * G, c = c0 + mine, row = first + c;
    if (first + c0 >= rows || rows <= pl.rows_lo || rows > pl.rows_hi) return;  // none of the workgroup's rows
    const float* wp = a.ws + (tile * a.Hkv + kvh) * pl.splits * PART;
    // the parts' maxima and sums, up to 256 / THREADS parts a thread
    float2 ml[SHARE];
    float M = -INFINITY;
#pragma unroll
    for (int i = 0; i < SHARE; ++i) {
        const int s = own + i * THREADS;
        ml[i] = make_float2(-INFINITY, 0.0f);
        if (s < pl.splits) ml[i] = *reinterpret_cast<const float2*>(wp + (int64_t)s * PART + BM * DP + 2 * c);
        M = fmaxf(M, ml[i].x);
    }
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) M = fmaxf(M, __shfl_xor(M, x));
    if (THREADS > 64) {
        if ((tid & 63) == 0) most[wave] = M;
        __syncthreads();
        M = fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3]));
    }
    const float Mc = M == -INFINITY ? 0.0f : M;
    float L = 0.0f;
#pragma unroll
    for (int i = 0; i < SHARE; ++i) {
        const float f = __builtin_amdgcn_exp2f(ml[i].x - Mc);  // 0 for a part that saw no key of the row
        factor[mine][own + i * THREADS] = f;
        L = __builtin_fmaf(f, ml[i].y, L);
    }
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) L += __shfl_xor(L, x);
    if (THREADS > 64 && (tid & 63) == 0) total[wave] = L;
    __syncthreads();
    if (THREADS > 64) L = (total[0] + total[1]) + (total[2] + total[3]);
    const int d = own % PER * 4, sub = own / PER;
    f32x4 acc = {0, 0, 0, 0};
    if (sub < SUBS)
        for (int s0 = sub; s0 < pl.splits; s0 += SUBS * AHEAD) {
            f32x4 v[AHEAD];
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                const int s = s0 + i * SUBS;
                v[i] = *reinterpret_cast<const f32x4*>(wp + (int64_t)(s < pl.splits ? s : 0) * PART + c * DP + d);
            }
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                const int s = s0 + i * SUBS;
                if (s < pl.splits) {
                    const float f = factor[mine][s];
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[e] = __builtin_fmaf(f, v[i][e], acc[e]);
                }
            }
        }
    if (SUBS > 1) {
        sums[tid] = acc;
        __syncthreads();
        if (sub == 0)
#pragma unroll
            for (int i = 1; i < SUBS; ++i) acc += sums[tid + i * PER];
    }
    if (sub != 0 || row >= rows) return;
    const bool none = L == 0.0f;
    const int64_t tk = w.t0 + row / G;
    const int head = kvh * G + row % G;
    if (d < a.D) {
        uint16_t b[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) b[e] = from_f32<F16>(none ? 0.0f : acc[e] / L);
        *reinterpret_cast<uint2*>(a.out + tk * a.o_tok + (int64_t)head * a.o_head + d) =
            make_uint2(b[0] | (uint32_t)b[1] << 16, b[2] | (uint32_t)b[3] << 16);
    }
    if (a.lse && d == 0) a.lse[tk * a.H + head] = none ? -INFINITY : (M + __log2f(L)) * LN2;
}

// ---------------------------------------------------------------------------------------------

struct Parts {
    int64_t few_tiles, many_tiles;
    int few_splits, many_splits;  // 0: not launched
    int few_waves;                // of a workgroup
    int many_each;                // Plan::each
};

int padded_dim(int D) { return D <= 64 ? 64 : D <= 96 ? 96 : D <= 128 ? 128 : D <= 192 ? 192 : 256; }
// That of few_rows_kernel: a lane's fourth of 96 microscaled values would go in pieces of 8, which at 128 are 32 (or 16).  64
// requests of up to 8,192 keys (24 heads over 8, D = 96), us in short runs, 96 | 128: MXFP8 186 | 158, MXFP4 161 | 105.
template <int KIND>
constexpr int few_dim(int padded) { return KIND != CACHE_16 && padded == 96 ? 128 : padded; }

int splits_for(int64_t groups, int64_t want, int max_kv, int least_keys) {
    int64_t s = groups < 1 ? 1 : want / groups, most = max_kv / least_keys;
    if (s > most) s = most;
    return s < 1 ? 1 : s > 256 ? 256 : (int)s;
}

Parts divide(int R, int T, int max_q, int max_kv, int H, int Hkv, int D, bool mx) {
    const int64_t G = H / Hkv, rows = max_q * G;
    Parts p{};
    p.few_waves = 4;
    p.few_tiles = R > 0 ? R : 1;
    if (rows <= FEW || (int64_t)R * max_q != T) {  // some requests may have few rows
        // A workgroup per CU, two up to 64 dimensions; D = 128 (64), us: 32 requests of 4,000 keys 31.0 (21.9) at 256
        // workgroups, 31.4 (19.3) at 512, 33.1 (19.6) at 768; 100 of 9,000: 166 (125), 193 (97), 192 (108).  64 keys at
        // least: one request of 1,000 keys 10.3 us, at 128 11.7, at 256 14.1.
        p.few_splits = splits_for(p.few_tiles * Hkv, D <= 64 ? 512 : 256, max_kv, 64);
        // Microscaled blocks, up to 768 keys: eight waves of one workgroup take all of a request's keys in one launch, where
        // that gives a wave not many more tiles than the parts do, whose join takes 3 to 4 us.  32 heads over 8, us in
        // graphs, 8 waves | parts, MXFP8 (MXFP4), pages of 16 tokens:
        //                          256 keys                    512                       768
        //   D =  64, 1 request    5.8 |  8.3 (5.6 |  8.3)   6.9 |  8.3 (6.8 |  8.2)   8.1 |  8.4 (7.9 |  8.4)
        //   D = 128, 1            7.3 |  8.9 (6.5 |  8.6)   9.5 |  9.0 (8.1 |  8.7)  11.6 |  9.3 (9.6 |  9.0)
        //            8            7.5 |  9.7 (6.7 |  9.4)   9.6 | 10.2 (8.3 |  9.5)  11.7 | 11.5 (9.8 | 10.6)
        //   D = 192, 1            8.3 |  9.7 (7.9 |  9.6)  10.6 | 10.1 (9.9 | 10.0)  13.6 | 10.2 (12.5 | 10.1)
        //   D = 256, 1           11.1 | 10.8 (8.7 |  9.8)  15.5 | 11.1 (11.1 | 10.3) 20.6 | 11.3 (13.5 | 10.5)
        //            16          11.2 | 13.7 (8.9 | 12.2)  17.6 | 18.1 (11.4 | 14.3) 22.9 | 22.4 (13.9 | 16.5)
        // Pages of 8 or 24 are within 10 % of these on both sides.  Called from Python, where parts cost an allocation and a
        // launch, 10.4 | 14.8 at D = 128 with 450 keys and 11.6 | 14.8 (10.4 | 14.8) with 768: up to 128 dimensions all 768
        // stay in one launch.
        if (mx && max_kv <= 768 && p.few_splits > 1) {
            const int parts = 128 * p.few_splits, more_tiles = (max_kv + 255) / 256 - (max_kv + parts - 1) / parts;  // a wave's
            if (more_tiles <= (D <= 128 ? 2 : D <= 192 ? 1 : 0)) {
                p.few_splits = 1;
                p.few_waves = 8;
            }
        }
    }
    if (rows > FEW && R > 0) {
        // Whichever numbering of the row tiles takes fewer: by the tokens in front of a request, or as many for each as
        // max_q allows (a step padded to far more tokens than its requests have: 8,192 tokens, one request of 32 at most,
        // 32 heads over 8: 8 tiles in place of 1,040, and 34 MB of workspace in place of 4.4 GB).
        const int64_t by_tokens = T * G / MANY + R + 1, each = (rows + MANY - 1) / MANY;
        p.many_each = R * each <= by_tokens ? (int)each : 0;
        p.many_tiles = p.many_each ? R * each : by_tokens;
        // A workgroup per CU and no more (D = 128): 32 requests of 16 tokens against 2,000 keys 56 us, at 512 workgroups 88;
        // 4 of 64 against 8,000 77 and 85.  Parts of 128 or 512 keys at least: the same within 1 %.
        p.many_splits = splits_for(p.many_tiles * Hkv, 256, max_kv, 256);
    }
    return p;
}

// Parts to add to a grid of `groups` workgroups a part, so that some 8 pieces a thread zero the tokens that cannot be a
// request's.  Where all may be one's, the grid has their rows to work on anyway.
unsigned parts_to_zero(const AttentionArgs& a, int64_t groups, int parts) {
    const int64_t spare = a.T - (int64_t)a.R * a.max_q;
    if (spare <= 0) return 0;
    int64_t want = spare * a.H * a.D / (8 * 8 * 256);
    if (want > 512) want = 512;
    const int64_t more = (want + groups - 1) / groups - parts;
    return more > 0 ? (unsigned)more : 0;
}

template <int KIND, bool F16, int DP>
hipError_t launch_dim(const AttentionArgs& a, Plan pl, const Parts& p, hipStream_t st) {
    pl.zero_rest = 1;
    if (p.few_splits) {
        pl.splits = p.few_splits;
        pl.rows_lo = 0;
        pl.rows_hi = FEW;
        pl.tiles = p.few_tiles;
        const unsigned more = parts_to_zero(a, p.few_tiles * a.Hkv, p.few_splits);
        const dim3 grid(a.Hkv, (unsigned)p.few_tiles, p.few_splits + more);
        constexpr int FP = few_dim<KIND>(DP);
        // 16 keys that start at a multiple of 16 are in one page: its place is worked out once for the wave, and a lane's share
        // of it is an offset of 32 bits.
        const bool page16 = KIND != CACHE_16 && a.page % 16 == 0 && (a.c_row | a.s_row) < 1 << 26;
        if constexpr (KIND != CACHE_16) {
            if (p.few_waves == 8 && page16)
                hipLaunchKernelGGL((few_rows_kernel<KIND, F16, FP, true, 8>), grid, dim3(512), 0, st, a, pl);
            else if (p.few_waves == 8)
                hipLaunchKernelGGL((few_rows_kernel<KIND, F16, FP, false, 8>), grid, dim3(512), 0, st, a, pl);
            else if (page16)
                hipLaunchKernelGGL((few_rows_kernel<KIND, F16, FP, true, 4>), grid, dim3(256), 0, st, a, pl);
        }
        if (!page16 && p.few_waves == 4)
            hipLaunchKernelGGL((few_rows_kernel<KIND, F16, FP, false, 4>), grid, dim3(256), 0, st, a, pl);
        if (p.few_splits > 1)
            hipLaunchKernelGGL((join_kernel<F16, FP, FEW, 256>), dim3((unsigned)(p.few_tiles * a.Hkv * FEW)), dim3(256), 0,
                               st, a, pl);
        pl.zero_rest = 0;
    }
    if (p.many_splits) {
        pl.splits = p.many_splits;
        pl.rows_lo = p.few_splits ? FEW : 0;
        pl.rows_hi = INT32_MAX;
        pl.tiles = p.many_tiles;
        pl.each = p.many_each;
        const unsigned more = pl.zero_rest ? parts_to_zero(a, p.many_tiles * a.Hkv, p.many_splits) : 0;
        hipLaunchKernelGGL((many_rows_kernel<KIND, F16, DP, (DP <= 128 ? 64 : 32)>),
                           dim3((unsigned)(p.many_tiles * a.Hkv), p.many_splits + more), dim3(2 * MANY), 0, st, a, pl);
        if (p.many_splits > 1)
            hipLaunchKernelGGL((join_kernel<F16, DP, MANY, 64>), dim3((unsigned)(p.many_tiles * a.Hkv * (MANY / 4))), dim3(256),
                               0, st, a, pl);
    }
    return hipGetLastError();
}

template <int KIND, bool F16>
hipError_t launch_type(const AttentionArgs& a, const Plan& pl, const Parts& p, hipStream_t st) {
    switch (padded_dim(a.D)) {
        case 64: return launch_dim<KIND, F16, 64>(a, pl, p, st);
        case 96: return launch_dim<KIND, F16, 96>(a, pl, p, st);
        case 128: return launch_dim<KIND, F16, 128>(a, pl, p, st);
        case 192: return launch_dim<KIND, F16, 192>(a, pl, p, st);
        default: return launch_dim<KIND, F16, 256>(a, pl, p, st);
    }
}

template <int KIND>
hipError_t launch_kind(const AttentionArgs& args, hipStream_t st) {
    AttentionArgs a = args;
    if (a.n_pages == 0) a.max_pages = 0;  // no key is read
    Plan pl{};
    pl.c = fmaxf(fabsf(a.scale) * 1.44269504f, 1e-37f);
    pl.flip = a.scale < 0.0f ? 0x80008000u : 0u;
    int bits = 0;
    while (((int64_t)1 << bits) < a.page) ++bits;
    pl.magic = (uint32_t)((((uint64_t)1 << (31 + bits)) + a.page - 1) / a.page);
    pl.shift = 31 + bits;
    pl.G = a.H / a.Hkv;
    const Parts p = divide(a.R, a.T, a.max_q, a.max_kv, a.H, a.Hkv, a.D, KIND != CACHE_16);
    return a.f16 ? launch_type<KIND, true>(a, pl, p, st) : launch_type<KIND, false>(a, pl, p, st);
}

}  // namespace
}  // namespace cqk
