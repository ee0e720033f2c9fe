// Arguments of the operators that run a packed checkpoint (linear layer, paged cache, attention).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace cqk {

// y [M][out] = act(x W + bias) + residual over GPTQ-v1 tensors; gated: W has 2 out columns, the
// gate's first, and y = act(gate) * up + residual.  Strides in elements.
struct LinearArgs {
    const uint16_t* x;
    const int32_t* qw;
    const uint16_t* scales;
    const uint16_t* bias;      // [out (* 2 if gated)] or null, of x's type
    const uint16_t* residual;  // [M][ldr] or null, of x's type
    void* y;
    int64_t M, out, in, ldx, ldr, ldy;
    int x_f16, y_f32, act, gated;
};
hipError_t launch_linear(const LinearArgs& a, hipStream_t st);

struct BlockMapArgs {
    const int32_t *ctx, *add, *free_pages, *n_free;
    int32_t* table;
    int32_t *cu, *kv_len, *slots, *positions, *status, *n_left;
    int64_t table_stride;
    int32_t R, page, free_cap, max_pages, max_tokens;
};
hipError_t launch_block_map(const BlockMapArgs& a, hipStream_t st);

// K and V rows [T][Hkv][D] into pages by slot; strides in elements, D contiguous.
struct CacheWriteArgs {
    const uint16_t *k, *v;
    uint16_t *kc, *vc;
    const int32_t* slots;
    int64_t k_tok, k_head, v_tok, v_head;
    int64_t c_page, c_head, c_row;
    int64_t n_slots;
    int32_t T, H, D, page;
};
hipError_t launch_cache_write(const CacheWriteArgs& a, hipStream_t st);

struct AttentionArgs {
    const uint16_t *q, *kc, *vc;
    uint16_t* out;
    float* lse;  // [T][H] or null
    const int32_t *table, *cu, *kv_len;
    int64_t q_tok, q_head, o_tok, o_head;
    int64_t c_page, c_head, c_row;
    int64_t table_stride;
    int32_t page, n_pages, max_pages;
    int32_t R, T, max_q, max_kv, H, Hkv, D, causal, window, f16;
    float scale;
    float* ws;
};
// Whether the grid for these sizes (its threads numbered in 32 bits) can be launched.
bool attention_fits(int32_t R, int32_t T, int32_t max_q, int32_t max_kv, int32_t H, int32_t Hkv, int32_t D);
// Floats of workspace the launch for these sizes uses (0: none).
int64_t attention_ws(int32_t R, int32_t T, int32_t max_q, int32_t max_kv, int32_t H, int32_t Hkv, int32_t D);
hipError_t launch_attention(const AttentionArgs& a, hipStream_t st);

}  // namespace cqk
