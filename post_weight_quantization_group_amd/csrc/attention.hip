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
// size of the output's own: relative to 64 bits the outputs are off by 2.1e-3 to 2.3e-3 (bf16; f16 2.5e-4), an fp32
// evaluation that is rounded at the end by 1.7e-3 (2.0e-4).
//
// A masked key has weight 0, and 0 times an infinity or a NaN in V would be a NaN: keys that no row
// of the tile sees are loaded as zeros, and where a tile's mask differs between its rows, what is not
// finite in its V is staged as 0 and read again, key by key, into two bits per output (an infinity of
// either sign seen; both: NaN) that are applied at the end.
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

// ---------------------------------------------------------------------------------------------
// Few rows (generation): a workgroup takes a request's rows (at most 16) and one part of the keys; its four waves take
// tiles of 32 keys in turn, each with its own running maximum, and join at the end.  Bound by reading K and V: both go
// from memory to registers in pieces of 16 bytes a lane, the next tile's while this one is worked on; V passes through
// the wave's own LDS to be transposed, so the waves never wait for each other.  64 requests of up to 8,192 keys (32
// heads over 8, D = 128): 323 us, 5.3 TB/s (a copy of 2 GiB reaches 4.9).  One request of some 400 keys: 7.2 us, of
// which three loads that wait for each other (lengths, table, keys) take the most, and 4.0 for the join.  D = 256 (one wave
// per SIMD): the same 64 requests 646 us, 5.3 TB/s.  Four waves a workgroup | eight, us: one request of 100 keys 6.5 | 6.6,
// at D = 256 8.7 | 11.4, the 64 requests at D = 256 646 | 757 (eight spill), at D = 128 and 64 the same.
template <bool F16, int DP>
__global__ __launch_bounds__(256) void few_rows_kernel(AttentionArgs a, Plan pl) {
    constexpr int BM = FEW, BN = 32, KS = DP / 32, DT = DP / 16;
    constexpr int VS = DP + ((DP / 2) % 64 == 16 || (DP / 2) % 64 == 48 ? 0 : 32);  // rows 16 banks apart (mod 64)
    constexpr int OS = DP + 4;
    constexpr int WAVE_BYTES = BN * VS * 2 > BM * OS * 4 ? BN * VS * 2 : BM * OS * 4;
    __shared__ __align__(16) uint8_t lds[4 * WAVE_BYTES];
    __shared__ float wave_m[4][BM], wave_l[4][BM];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, col = lane & 15, quad = lane >> 4;
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

    int64_t q_at = (int64_t)(w.t0 + tok) * a.q_tok + (int64_t)(kvh * G + row - tok * G) * a.q_head + 8 * quad;
    asm volatile("" : "+v"(q_at));  // worked out once, and not in front of every load
    s16x8 q[KS];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (live && 32 * ks + 8 * quad < a.D) {
            v = *reinterpret_cast<const uint4*>(a.q + q_at + 32 * ks);
            v.x ^= pl.flip; v.y ^= pl.flip; v.z ^= pl.flip; v.w ^= pl.flip;
        }
        q[ks] = __builtin_bit_cast(s16x8, v);
    }

    // this part's tiles of 32 keys
    const int t_begin = w.key_begin / BN, t_end = (w.key_end + BN - 1) / BN;
    const int per = max(0, (t_end - t_begin + pl.splits - 1) / pl.splits);
    const int t0 = t_begin + split * per, t1 = min(t_end, t0 + per);
    const int32_t* table = a.table + r * a.table_stride;

    int page_id[2];
    auto fetch_ids = [&](int t) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int key = t * BN + 16 * h + col;
            page_id[h] = -1;
            if (t < t1 && key >= w.key_begin && key < w.key_end) page_id[h] = table[page_of(pl, key)];
        }
    };
    uint4 kr[2][KS], vr[2][KS];
    int ok_next[2];
    auto fetch_kv = [&](int t) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int key = t * BN + 16 * h + col;
            ok_next[h] = page_id[h] >= 0 && page_id[h] < a.n_pages;
            const int64_t at = page_id[h] * a.c_page + kvh * a.c_head + (int64_t)(key - page_of(pl, key) * a.page) * a.c_row + 8 * quad;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) kr[h][ks] = vr[h][ks] = make_uint4(0, 0, 0, 0);
            if (!ok_next[h]) continue;
            if (a.D == DP) {
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) kr[h][ks] = *reinterpret_cast<const uint4*>(a.kc + at + 32 * ks);
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) vr[h][ks] = *reinterpret_cast<const uint4*>(a.vc + at + 32 * ks);
            } else {
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
                    if (32 * ks + 8 * quad < a.D) {
                        kr[h][ks] = *reinterpret_cast<const uint4*>(a.kc + at + 32 * ks);
                        vr[h][ks] = *reinterpret_cast<const uint4*>(a.vc + at + 32 * ks);
                    }
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
    fetch_ids(t + 4);
    for (; t < t1; t += 4) {
        f32x4 s[2];
        const bool mixed = t * BN < same_lo || (t + 1) * BN > same_hi;
        uint64_t there[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            s[h] = f32x4{0, 0, 0, 0};
            there[h] = __ballot(ok_next[h]);
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                s[h] = mfma16<F16>(__builtin_bit_cast(s16x8, kr[h][ks]), q[ks], s[h]);
                *reinterpret_cast<uint4*>(vl + (16 * h + col) * VS + 32 * ks + 8 * quad) = vr[h][ks];
            }
        }
        bool special = false;
        if (mixed) {
            u16x2 most = {0, 0};
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) most = largest_exponents<F16>(most, vr[h][ks]);
            special = __any(not_finite<F16>(most.x) || not_finite<F16>(most.y));
            if (special)
#pragma unroll 1
                for (int i = quad; i < 2 * DP / 8; i += 4) {  // the pieces this lane has stored
                    uint4* at = reinterpret_cast<uint4*>(vl + (16 * (i / (DP / 8)) + col) * VS + 8 * (i % (DP / 8)));
                    *at = finite_part<F16>(*at);
                }
        }
        fetch_kv(t + 4);
        fetch_ids(t + 8);
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
                const uint16_t* v = a.vc + id * a.c_page + kvh * a.c_head + (int64_t)(key - page_of(pl, key) * a.page) * a.c_row;
                if (key >= see_lo && key < see_hi)  // (also where its weight is 0)
#pragma unroll 1
                    for (int d = 0; d < DT; ++d)
                        if (16 * d + 4 * quad < a.D) seen.template add<F16>(d, *reinterpret_cast<const uint2*>(v + 16 * d + 4 * quad));
            }
        }
    }
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);

    // join the four waves
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
    for (int i = tid; i < live_rows * (DP / 4); i += 256) {
        const int c = i / (DP / 4), d = i % (DP / 4) * 4;
        float M = -INFINITY;
#pragma unroll
        for (int x = 0; x < 4; ++x) M = fmaxf(M, wave_m[x][c]);
        const float Mc = M == -INFINITY ? 0.0f : M * pl.c;
        float L = 0.0f;
        f32x4 acc = {0, 0, 0, 0};
#pragma unroll
        for (int x = 0; x < 4; ++x) {
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
template <bool F16, int DP, int BN>
__global__ __launch_bounds__(2 * MANY, 2) void many_rows_kernel(AttentionArgs a, Plan pl) {
    constexpr int BM = MANY, KS = DP / 16, DT = DP / 32, KT = BN / 32;
    constexpr int RUNS = BN * DP / 8 / 64, WAVES = MANY / 32;  // loads of 64 16-byte pieces a tile of K or V takes
    constexpr int PIECES = (RUNS + WAVES - 1) / WAVES;         // of them, per wave
    constexpr int STAGES = 4, BLOCK = 2 * MANY;  // tiles in LDS; keys looked up at a time, one per thread
    __shared__ __align__(256) uint16_t ktile[STAGES][BN * DP];
    __shared__ __align__(256) uint16_t vtile[STAGES][BN * DP];
    __shared__ int64_t row_at[2][BLOCK];             // of block b, in [b % 2]: offset of each key's row, -1: none
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

    // Where the rows of a block of keys lie, a thread per key: find() starts the table's load, note() ends it.
    auto find = [&](int b) {
        const int key = b * BLOCK + tid;
        return key >= t0 * BN && key < t1 * BN && key >= w.key_begin && key < w.key_end ? table[page_of(pl, key)] : INT32_MIN;
    };
    auto note = [&](int b, int id) {
        const int key = b * BLOCK + tid;
        const bool ok = id >= 0 && id < a.n_pages;
        row_at[b & 1][tid] = ok ? id * a.c_page + (int64_t)(key - page_of(pl, key) * a.page) * a.c_row : -1;
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
        for (int t = t0; t < min(t0 + STAGES - 1, t1); ++t) fetch(t);
    }
    for (int t = t0; t < t1; ++t) {
        // the two tiles after this one may still be on their way
        if (t + STAGES - 2 < t1) loaded_to_lds<(STAGES - 2) * 2 * (RUNS / WAVES)>();
        else loaded_to_lds<0>();
        __syncthreads();  // this tile is in LDS, the previous one has been read
        int id = INT32_MIN;
        const bool turn_over = t * BN % BLOCK == 0;  // the block before this one is done with
        if (turn_over) id = find(t * BN / BLOCK + 1);
        if (t + STAGES - 1 < t1) fetch(t + STAGES - 1);
        if (tid == 0) bad_at[(t + 2) & 3] = 0;
        bool special = false;
        if (t * BN < same_lo || (t + 1) * BN > same_hi) {  // the rows' masks differ here
#pragma unroll 1
            for (int i = 64 * wave + lane; i < 64 * RUNS; i += 64 * WAVES) {
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
        // four operands ahead of their products (the compiler reads each just before it)
        __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);
#pragma unroll
        for (int x = 0; x < KS * KT / 2 - 2; ++x) {
            __builtin_amdgcn_sched_group_barrier(0x8, 2, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x8, 4, 0);
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
                const uint16_t* v = a.vc + page * a.c_page + kvh * a.c_head + (int64_t)(key - page_of(pl, key) * a.page) * a.c_row;
                if (key >= see_lo && key < see_hi)  // (also where its weight is 0)
#pragma unroll 1
                    for (int j = 0; j < 4 * DT; ++j)  // accumulators 4 j .. of the lane: d = 8 j + 4 half ..
                        if (8 * j + 4 * half < a.D) seen.template add<F16>(j, *reinterpret_cast<const uint2*>(v + 8 * j + 4 * half));
            }
            seen_at[tid] = seen;
        }
        }
        if (turn_over) note(t * BN / BLOCK + 1, id);
    }
    l += __shfl_xor(l, 32);
    if (pl.splits > 1) {
        float* wp = a.ws + ((tile * a.Hkv + kvh) * pl.splits + split) * (BM * (DP + 2));
        const int c = 32 * wave + col;
        if (live) {
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int e = 0; e < 16; e += 4)
                    *reinterpret_cast<f32x4*>(wp + c * DP + 32 * d + 2 * e + 4 * half) =
                        f32x4{o[d][e], o[d][e + 1], o[d][e + 2], o[d][e + 3]};
            if (half == 0) {
                wp[BM * DP + 2 * c] = m * pl.c;
                wp[BM * DP + 2 * c + 1] = l;
            }
            if (seen_yet) seen_at[tid].apply([&](int i, float x) { wp[c * DP + 2 * (i & ~3) + 4 * half + (i & 3)] += x; });
        }
        return;
    }
    if (live) {
        const bool none = l == 0.0f;
        const float inv = none ? 0.0f : 1.0f / l;  // (o is 0 there)
        int64_t o_at = (int64_t)(w.t0 + tok) * a.o_tok + (int64_t)head * a.o_head + 4 * half;
        asm volatile("" : "+v"(o_at));
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int e = 0; e < 16; e += 4)
                if (32 * d + 2 * e + 4 * half < a.D) {
                    uint32_t b[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x) b[x] = from_f32<F16>(o[d][e + x] * inv);
                    *reinterpret_cast<uint2*>(a.out + o_at + 32 * d + 2 * e) = make_uint2(b[0] | b[1] << 16, b[2] | b[3] << 16);
                }
        if (seen_yet)
            seen_at[tid].apply([&](int i, float x) {
                if (2 * (i & ~3) + 4 * half >= a.D) return;
                uint16_t* at = a.out + o_at + 2 * (i & ~3) + (i & 3);
                *at = from_f32<F16>(to_f32<F16>(*at) + x);
            });
        if (a.lse && half == 0) a.lse[(int64_t)(w.t0 + tok) * a.H + head] = none ? -INFINITY : (m * pl.c + __log2f(l)) * LN2;
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
    int many_each;                // Plan::each
};

int padded_dim(int D) { return D <= 64 ? 64 : D <= 96 ? 96 : D <= 128 ? 128 : D <= 192 ? 192 : 256; }

int splits_for(int64_t groups, int64_t want, int max_kv, int least_keys) {
    int64_t s = groups < 1 ? 1 : want / groups, most = max_kv / least_keys;
    if (s > most) s = most;
    return s < 1 ? 1 : s > 256 ? 256 : (int)s;
}

Parts divide(int R, int T, int max_q, int max_kv, int H, int Hkv, int D) {
    const int64_t G = H / Hkv, rows = max_q * G;
    Parts p{};
    p.few_tiles = R > 0 ? R : 1;
    if (rows <= FEW || (int64_t)R * max_q != T) {  // some requests may have few rows
        // A workgroup per CU, two up to 64 dimensions; D = 128 (64), us: 32 requests of 4,000 keys 31.0 (21.9) at 256
        // workgroups, 31.4 (19.3) at 512, 33.1 (19.6) at 768; 100 of 9,000: 166 (125), 193 (97), 192 (108).  64 keys at
        // least: one request of 1,000 keys 10.3 us, at 128 11.7, at 256 14.1.
        p.few_splits = splits_for(p.few_tiles * Hkv, D <= 64 ? 512 : 256, max_kv, 64);
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

template <bool F16, int DP>
hipError_t launch_dim(const AttentionArgs& a, Plan pl, const Parts& p, hipStream_t st) {
    pl.zero_rest = 1;
    if (p.few_splits) {
        pl.splits = p.few_splits;
        pl.rows_lo = 0;
        pl.rows_hi = FEW;
        pl.tiles = p.few_tiles;
        const unsigned more = parts_to_zero(a, p.few_tiles * a.Hkv, p.few_splits);
        hipLaunchKernelGGL((few_rows_kernel<F16, DP>), dim3(a.Hkv, (unsigned)p.few_tiles, p.few_splits + more), dim3(256),
                           0, st, a, pl);
        if (p.few_splits > 1)
            hipLaunchKernelGGL((join_kernel<F16, DP, FEW, 256>), dim3((unsigned)(p.few_tiles * a.Hkv * FEW)), dim3(256), 0,
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
        hipLaunchKernelGGL((many_rows_kernel<F16, DP, (DP <= 128 ? 64 : 32)>),
                           dim3((unsigned)(p.many_tiles * a.Hkv), p.many_splits + more), dim3(2 * MANY), 0, st, a, pl);
        if (p.many_splits > 1)
            hipLaunchKernelGGL((join_kernel<F16, DP, MANY, 64>), dim3((unsigned)(p.many_tiles * a.Hkv * (MANY / 4))), dim3(256),
                               0, st, a, pl);
    }
    return hipGetLastError();
}

template <bool F16>
hipError_t launch_type(const AttentionArgs& a, const Plan& pl, const Parts& p, hipStream_t st) {
    switch (padded_dim(a.D)) {
        case 64: return launch_dim<F16, 64>(a, pl, p, st);
        case 96: return launch_dim<F16, 96>(a, pl, p, st);
        case 128: return launch_dim<F16, 128>(a, pl, p, st);
        case 192: return launch_dim<F16, 192>(a, pl, p, st);
        default: return launch_dim<F16, 256>(a, pl, p, st);
    }
}

}  // namespace

bool attention_fits(int32_t R, int32_t T, int32_t max_q, int32_t max_kv, int32_t H, int32_t Hkv, int32_t D) {
    return divide(R, T, max_q, max_kv, H, Hkv, D).many_tiles * Hkv <= UINT32_MAX / (2 * MANY);
}

int64_t attention_ws(int32_t R, int32_t T, int32_t max_q, int32_t max_kv, int32_t H, int32_t Hkv, int32_t D) {
    const Parts p = divide(R, T, max_q, max_kv, H, Hkv, D);
    const int64_t row = padded_dim(D) + 2;
    const int64_t few = p.few_splits > 1 ? p.few_tiles * Hkv * p.few_splits * FEW * row : 0;
    const int64_t many = p.many_splits > 1 ? p.many_tiles * Hkv * p.many_splits * MANY * row : 0;
    return few > many ? few : many;
}

hipError_t launch_attention(const AttentionArgs& args, hipStream_t st) {
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
    const Parts p = divide(a.R, a.T, a.max_q, a.max_kv, a.H, a.Hkv, a.D);
    return a.f16 ? launch_type<true>(a, pl, p, st) : launch_type<false>(a, pl, p, st);
}

}  // namespace cqk
