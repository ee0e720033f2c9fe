// Attention over a paged cache of 16-bit values.
#include "attention.h"

namespace cqk {

bool attention_fits(int32_t R, int32_t T, int32_t max_q, int32_t max_kv, int32_t H, int32_t Hkv, int32_t D) {
    return divide(R, T, max_q, max_kv, H, Hkv, D, false).many_tiles * Hkv <= UINT32_MAX / (2 * MANY);
}

int64_t attention_ws(int32_t R, int32_t T, int32_t max_q, int32_t max_kv, int32_t H, int32_t Hkv, int32_t D, bool mx) {
    const Parts p = divide(R, T, max_q, max_kv, H, Hkv, D, mx);
    const int64_t row = padded_dim(D) + 2, few_row = (mx ? few_dim<MXFP4>(padded_dim(D)) : padded_dim(D)) + 2;
    const int64_t few = p.few_splits > 1 ? p.few_tiles * Hkv * p.few_splits * FEW * few_row : 0;
    const int64_t many = p.many_splits > 1 ? p.many_tiles * Hkv * p.many_splits * MANY * row : 0;
    return few > many ? few : many;
}

hipError_t launch_attention(const AttentionArgs& a, hipStream_t st) { return launch_kind<CACHE_16>(a, st); }

}  // namespace cqk
