// Attention of new tokens over a paged cache, the simple form: a wave per (token, head), its lanes
// over the head's dimensions.
#include "serve_args.h"
#include "serve_math.h"

namespace cqk {
namespace {

template <bool F16>
__global__ __launch_bounds__(64) void attention_kernel(AttentionArgs a) {
    const int t = blockIdx.x, h = blockIdx.y, lane = threadIdx.x;
    int lo = 0, hi = a.R;  // the request with cu[r] <= t < cu[r + 1]
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (a.cu[mid + 1] > t) hi = mid;
        else lo = mid + 1;
    }
    const bool mine = lo < a.R && a.cu[lo] <= t;
    float acc[4] = {0, 0, 0, 0}, q[4] = {0, 0, 0, 0}, m = -INFINITY, l = 0.0f;
    for (int i = 0; i < 4; ++i)
        if (lane + 64 * i < a.D) q[i] = to_f32<F16>(a.q[t * a.q_tok + h * a.q_head + lane + 64 * i]);
    if (mine) {
        const int n = a.cu[lo + 1] - a.cu[lo];
        const int64_t room = (int64_t)a.max_pages * a.page;
        const int64_t kv = a.kv_len[lo] < room ? a.kv_len[lo] : room;
        const int64_t p = kv - n + (t - a.cu[lo]);
        int64_t end = kv, begin = 0;
        if (a.causal && p + 1 < end) end = p + 1;
        if (a.window && p - a.window + 1 > begin) begin = p - a.window + 1;
        for (int64_t j = begin; j < end; ++j) {
            const int pg = a.table[lo * a.table_stride + j / a.page];
            if (pg < 0 || pg >= a.n_pages) continue;
            const int64_t at = pg * a.c_page + (h / (a.H / a.Hkv)) * a.c_head + j % a.page * a.c_row;
            float s = 0.0f;
            for (int i = 0; i < 4; ++i)
                if (lane + 64 * i < a.D) s = __builtin_fmaf(q[i], to_f32<F16>(a.kc[at + lane + 64 * i]), s);
            for (int x = 32; x; x >>= 1) s += __shfl_xor(s, x);
            s *= a.scale;
            const float top = fmaxf(m, s);
            const float keep = __expf(m - top), e = __expf(s - top);
            l = l * keep + e;
            for (int i = 0; i < 4; ++i)
                if (lane + 64 * i < a.D) acc[i] = acc[i] * keep + e * to_f32<F16>(a.vc[at + lane + 64 * i]);
            m = top;
        }
    }
    for (int i = 0; i < 4; ++i)
        if (lane + 64 * i < a.D) a.out[t * a.o_tok + h * a.o_head + lane + 64 * i] = from_f32<F16>(l > 0.0f ? acc[i] / l : 0.0f);
    if (a.lse && lane == 0) a.lse[(int64_t)t * a.H + h] = l > 0.0f ? m + __logf(l) : -INFINITY;
}

}  // namespace

int64_t attention_ws(int32_t, int32_t, int32_t, int32_t, int32_t, int32_t, int32_t) { return 0; }

hipError_t launch_attention(const AttentionArgs& a, hipStream_t st) {
    const dim3 grid((unsigned)a.T, (unsigned)a.H);
    if (a.f16) hipLaunchKernelGGL(attention_kernel<true>, grid, dim3(64), 0, st, a);
    else hipLaunchKernelGGL(attention_kernel<false>, grid, dim3(64), 0, st, a);
    return hipGetLastError();
}

}  // namespace cqk
