// The paged key/value cache of a packed checkpoint's run: block tables and slot maps from request
// lengths, and the writing of new keys and values into the pages.
#include "serve_args.h"

namespace cqk {
namespace {

constexpr int MAP_THREADS = 1024;

// Sums that stay at their largest value instead of wrapping: all that is asked of them is whether they
// exceed a limit below 2^31.
__device__ __forceinline__ uint32_t add_sat(uint32_t x, uint32_t y) { return __builtin_elementwise_add_sat(x, y); }
// Inclusive sums over the lanes of a wave: within rows of 16 lanes by shifts, then row ends onto the rows behind.
__device__ __forceinline__ uint32_t scan_of_wave(uint32_t x) {
    x = add_sat(x, __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, false));  // row_shr:1
    x = add_sat(x, __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, false));
    x = add_sat(x, __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, false));
    x = add_sat(x, __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, false));
    x = add_sat(x, __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false));  // lane 15 (47) to the second (fourth) row
    return add_sat(x, __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false));  // lane 31 to the upper rows
}
__device__ __forceinline__ uint32_t pages_for(int32_t tokens, int32_t page) {
    return (uint32_t)tokens / (uint32_t)page + ((uint32_t)tokens % (uint32_t)page != 0);
}

// Block tables and slot maps.  Request r holds ctx_r tokens and receives add_r more:
//   need_r = ceil((ctx_r + add_r) / page) - ceil(ctx_r / page) pages, 0 for an invalid request;
//   P_r, C_r = inclusive prefix sums of need and add over the valid requests;
//   r is served iff it is valid, P_r <= n_free and C_r <= max_tokens (both sums only grow, so the
//   served requests are the valid ones before the first that does not fit);
//   its i-th new page is free_pages[n_free - 1 - (P_r - need_r) - i], and the token at position p
//   has the slot table[r][p / page] * page + p % page.
// Integers only: the bound is the latency of one launch and of the chain load - scan - search -
// store.  Every workgroup therefore scans all requests by itself (8 bytes each, out of L2) instead
// of waiting for another launch, and then serves its own share of the tokens (binary search in the
// scan, in LDS) and of the table's new entries.  8 requests: 3.2 us; 512 requests with 105,000 tokens in 103
// workgroups: 5.6 us.
__global__ __launch_bounds__(MAP_THREADS) void block_map_kernel(BlockMapArgs a) {
    extern __shared__ int32_t lds[];
    int32_t* cum = lds;               // [R] served tokens through r (C_r, frozen from the first misfit on)
    int32_t* first = lds + a.R;       // [R] pages taken before r; -1 - that for a request not served
    __shared__ uint32_t wave_pages[MAP_THREADS / 64], wave_tokens[MAP_THREADS / 64];
    __shared__ int32_t served_pages, served_tokens;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int32_t n_free = a.n_free[0];
    n_free = n_free < 0 ? 0 : n_free > a.free_cap ? a.free_cap : n_free;
    if (tid == 0) served_pages = served_tokens = 0;
    uint32_t base_pages = 0, base_tokens = 0;
    for (int r0 = 0; r0 < a.R; r0 += MAP_THREADS) {
        const int r = r0 + tid;
        uint32_t need = 0, add = 0;
        int32_t ctx = 0;
        bool valid = false;
        if (r < a.R) {
            ctx = a.ctx[r];
            const int32_t n = a.add[r];
            valid = ctx >= 0 && n >= 0 && (int64_t)ctx + n <= (int64_t)a.max_pages * a.page;
            if (valid) {
                add = n;
                need = pages_for(ctx + n, a.page) - pages_for(ctx, a.page);
            }
        }
        uint32_t p = scan_of_wave(need), c = scan_of_wave(add);
        if (r0 > 0) __syncthreads();  // the wave sums of the previous 1,024 requests have been read
        if (lane == 63) {
            wave_pages[wave] = p;
            wave_tokens[wave] = c;
        }
        __syncthreads();
        const int waves = min(MAP_THREADS, a.R - r0 + 63) / 64;  // that hold requests
        uint32_t all_p = base_pages, all_c = base_tokens;
        for (int w = 0; w < waves; ++w) {
            if (w == wave) {
                p = add_sat(p, all_p);
                c = add_sat(c, all_c);
            }
            all_p = add_sat(all_p, wave_pages[w]);
            all_c = add_sat(all_c, wave_tokens[w]);
        }
        base_pages = all_p;
        base_tokens = all_c;
        const bool fits = r < a.R && p <= (uint32_t)n_free && c <= (uint32_t)a.max_tokens;
        if (r < a.R) {
            const bool served = valid && fits;
            cum[r] = fits ? (int32_t)c : INT32_MAX;
            first[r] = served ? (int32_t)(p - need) : -1;
            if (blockIdx.x == 0) {
                a.status[r] = !valid ? 2 : fits ? 0 : 1;
                a.kv_len[r] = served ? (int32_t)(ctx + add) : ctx < 0 ? 0 : ctx;
            }
        }
        // the requests that fit are the first ones: the last of them holds the served sums
        if (lane == (int)__popcll(__ballot(fits)) - 1) {
            atomicMax(&served_pages, (int32_t)p);
            atomicMax(&served_tokens, (int32_t)c);
        }
    }
    __syncthreads();
    const int32_t total = served_tokens;
    if (blockIdx.x == 0) {
        for (int r = tid; r < a.R; r += MAP_THREADS) a.cu[r + 1] = cum[r] < total ? cum[r] : total;
        if (tid == 0) {
            a.cu[0] = 0;
            a.n_left[0] = n_free - served_pages;
        }
    }
    // new entries of the block tables, a wave per request
    for (int r = blockIdx.x * (MAP_THREADS / 64) + wave; r < a.R; r += gridDim.x * (MAP_THREADS / 64)) {
        const int32_t before = first[r];
        if (before < 0) continue;
        const int64_t ctx = a.ctx[r], end = ctx + a.add[r];
        const int64_t b0 = (ctx + a.page - 1) / a.page, b1 = (end + a.page - 1) / a.page;
        for (int64_t b = b0 + lane; b < b1; b += 64)
            a.table[r * a.table_stride + b] = a.free_pages[n_free - 1 - before - (b - b0)];
    }
    // the tokens' slots
    for (int64_t t = (int64_t)blockIdx.x * MAP_THREADS + tid; t < a.max_tokens; t += (int64_t)gridDim.x * MAP_THREADS) {
        int32_t slot = -1, pos = 0;
        if (t < total) {
            int lo = 0, hi = a.R - 1;  // the first request whose cumulative count exceeds t
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (cum[mid] > t) hi = mid;
                else lo = mid + 1;
            }
            const int32_t ctx = a.ctx[lo];
            pos = ctx + (int32_t)(t - (lo > 0 ? cum[lo - 1] : 0));
            const int32_t b = pos / a.page, b0 = pages_for(ctx, a.page);
            const int32_t pg = b < b0 ? a.table[lo * a.table_stride + b]
                                      : a.free_pages[n_free - 1 - first[lo] - (b - b0)];
            const int64_t s = (int64_t)pg * a.page + pos % a.page;
            slot = pg < 0 || s > INT32_MAX ? -1 : (int32_t)s;
        }
        a.slots[t] = slot;
        a.positions[t] = pos;
    }
}

// Copy of K and V rows into their pages: a thread per 16 bytes (V = 8 elements) or per element.
// A copy: 4 T Hkv D bytes read and as many written bound it.  16,384 tokens of 8 heads of 128: 28.6 us, 4.7 TB/s (a copy
// of 2 GiB reaches 4.9); 64 tokens: 2.9 us.
template <int V>
__global__ __launch_bounds__(256) void cache_write_kernel(CacheWriteArgs a) {
    typedef uint16_t vec __attribute__((ext_vector_type(V)));
    const int64_t per_row = a.D / V, per_tok = per_row * a.H, n = per_tok * a.T;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t t = i / per_tok, rest = i % per_tok, h = rest / per_row, d = rest % per_row * V;
        const int64_t slot = a.slots[t];
        if (slot < 0 || slot >= a.n_slots) continue;
        const int64_t to = slot / a.page * a.c_page + h * a.c_head + slot % a.page * a.c_row + d;
        if constexpr (V == 1) {
            a.kc[to] = a.k[t * a.k_tok + h * a.k_head + d];
            a.vc[to] = a.v[t * a.v_tok + h * a.v_head + d];
        } else {
            *reinterpret_cast<vec*>(a.kc + to) = *reinterpret_cast<const vec*>(a.k + t * a.k_tok + h * a.k_head + d);
            *reinterpret_cast<vec*>(a.vc + to) = *reinterpret_cast<const vec*>(a.v + t * a.v_tok + h * a.v_head + d);
        }
    }
}

}  // namespace

hipError_t launch_block_map(const BlockMapArgs& a, hipStream_t st) {
    int64_t blocks = ((int64_t)a.max_tokens + MAP_THREADS - 1) / MAP_THREADS;
    const int64_t for_tables = (a.R + MAP_THREADS / 64 - 1) / (MAP_THREADS / 64);
    if (blocks < for_tables) blocks = for_tables;
    if (blocks > 256) blocks = 256;
    if (blocks < 1) blocks = 1;
    hipLaunchKernelGGL(block_map_kernel, dim3((unsigned)blocks), dim3(MAP_THREADS), (size_t)a.R * 8, st, a);
    return hipGetLastError();
}

hipError_t launch_cache_write(const CacheWriteArgs& a, hipStream_t st) {
    const int64_t strides = a.k_tok | a.k_head | a.v_tok | a.v_head | a.c_page | a.c_head | a.c_row | a.D;
    const uintptr_t ptrs = (uintptr_t)a.k | (uintptr_t)a.v | (uintptr_t)a.kc | (uintptr_t)a.vc;
    const int V = strides % 8 == 0 && ptrs % 16 == 0 ? 8 : 1;
    int64_t blocks = ((int64_t)a.T * a.H * (a.D / V) + 255) / 256;
    if (blocks > 16384) blocks = 16384;
    if (V == 8)
        hipLaunchKernelGGL(cache_write_kernel<8>, dim3((unsigned)blocks), dim3(256), 0, st, a);
    else
        hipLaunchKernelGGL(cache_write_kernel<1>, dim3((unsigned)blocks), dim3(256), 0, st, a);
    return hipGetLastError();
}

}  // namespace cqk
