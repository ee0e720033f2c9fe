// C ABI of the scale-selection library: argument checks, workspace carving,
// and kernel launches on the caller's stream.  Declared in include/cq.h.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <stddef.h>

#include "cq.h"
#include "launch.h"
#include "serve_args.h"

namespace {

constexpr size_t ALIGN = 256;
inline size_t round_up(size_t x) { return (x + ALIGN - 1) / ALIGN * ALIGN; }
inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
inline int32_t hip_status(hipError_t e) { return e == hipSuccess ? CQ_OK : CQ_EHIP; }

// Full-grid workspace: [counter | pad][int32 queue of n_groups]
size_t full_ws(int64_t n) { return ALIGN + round_up((size_t)n * 4u); }
// Bounded-sweep workspace: [counter | pad][int32 queue of n_groups][slice parts]
size_t sweep_ws(int64_t n) { return full_ws(n) + round_up(sizeof(cqk::SlicePart) * cqk::SLICE_PARTS); }
// Candidate workspace: [tie counter | pad][int32 tie list][sweep workspace]
size_t cand_ws(int64_t n) { return ALIGN + round_up((size_t)n * 4u) + sweep_ws(n); }

bool groups_ok(const float* w, const float* d, int64_t d_period, int32_t E, int64_t n_groups, size_t align = 16) {
    if (n_groups < 0 || E < 1 || E > CQ_MAX_ENVS) return false;
    if (n_groups == 0) return true;
    if (!w || !d || d_period < 1) return false;
    return aligned(w, align) && aligned(d, align);
}

bool spec_ok(int32_t G, int32_t qmin, int32_t qmax) {
    return G >= 1 && G <= CQ_MAX_GROUP && qmin >= -128 && qmin <= 0 && qmax >= 0 && qmax <= 127 && qmin < qmax;
}

// Quantizers the candidate solver takes besides the pages' own: at most 8 codes on each side of
// zero (8 transition slots per weight) and groups of at most 128 weights.
bool cand_spec_ok(int32_t G, int32_t qmin, int32_t qmax) { return G <= CQ_GROUP && qmin >= -8 && qmax <= 8; }

int32_t run_fullgrid(const float* w, const float* d, int32_t G, int32_t qmin, int32_t qmax, int64_t d_period, int32_t E,
                     int64_t n_groups, uint16_t* scales, int8_t* codes, double* objective, uint8_t* flags,
                     uint16_t* pooled_scales, double* pooled_objective, int want_minimax, uint8_t* ws,
                     hipStream_t st) {
    cqk::FullArgs a{};
    a.w = w; a.d = d; a.d_period = d_period; a.G = G; a.qmin = qmin; a.qmax = qmax;
    a.ratio = cqk::fullgrid_ratio(G, qmin, qmax, E);
    a.scales = scales; a.codes = codes; a.objective = objective; a.flags = flags;
    a.pscales = pooled_scales; a.pobjective = pooled_objective;
    a.want_minimax = want_minimax;
    a.want_pooled = (pooled_scales || pooled_objective) ? 1 : 0;
    a.fb_count = (int32_t*)ws;
    a.fb_list = (int32_t*)(ws + ALIGN);
    a.parts = (cqk::SlicePart*)(ws + full_ws(n_groups));  // the workspace is sweep_ws(n_groups) bytes
    return hip_status(cqk::launch_fullgrid(a, E, n_groups, st));
}

}  // namespace

extern "C" {

int32_t cq_abi_version(void) { return CQ_ABI_VERSION; }

const char* cq_status_string(int32_t s) {
    switch (s) {
        case CQ_OK: return "ok";
        case CQ_EINVAL: return "invalid argument";
        case CQ_EWORKSPACE: return "workspace missing, misaligned or too small";
        case CQ_EHIP: return "HIP launch failed";
        case CQ_EUNSUPPORTED: return "not supported by this entry point";
        case CQ_ELIMIT: return "more groups than the fixed scratch of the no-allocation entry point holds";
        default: return "unknown status";
    }
}

size_t cq_workspace_size(int32_t method, int32_t E, int64_t n_groups) {
    if (E < 1 || E > CQ_MAX_ENVS || n_groups < 0) return 0;
    // the full grid needs less than the bounded sweep; one size serves both, and the pooled
    // baseline (a bounded sweep) accepts the CQ_EXHAUSTIVE size too
    if (method == CQ_EXHAUSTIVE || method == CQ_BOUNDED) return sweep_ws(n_groups);
    if (method == CQ_CANDIDATE) return cand_ws(n_groups);
    return 0;
}

int32_t cq_quantize_groups(const float* w, const float* d, int64_t d_period, int32_t E, int64_t n_groups,
                           int32_t method, uint16_t* scales, int8_t* codes, double* objective, uint8_t* flags,
                           uint16_t* pooled_scales, double* pooled_objective, void* workspace,
                           size_t workspace_bytes, void* stream) {
    if (!groups_ok(w, d, d_period, E, n_groups)) return CQ_EINVAL;
    if (method != CQ_EXHAUSTIVE && method != CQ_CANDIDATE && method != CQ_BOUNDED) return CQ_EINVAL;
    if (n_groups > 0 && !scales) return CQ_EINVAL;
    if (n_groups > INT32_MAX) return CQ_EINVAL;
    if (method == CQ_CANDIDATE && (pooled_scales || pooled_objective)) return CQ_EUNSUPPORTED;
    if (n_groups == 0) return CQ_OK;
    const size_t need = cq_workspace_size(method, E, n_groups);
    if (!workspace || workspace_bytes < need || !aligned(workspace, ALIGN)) return CQ_EWORKSPACE;
    hipStream_t st = (hipStream_t)stream;
    uint8_t* ws = (uint8_t*)workspace;
    if (method == CQ_EXHAUSTIVE)
        return run_fullgrid(w, d, CQ_GROUP, -8, 7, d_period, E, n_groups, scales, codes, objective, flags,
                            pooled_scales, pooled_objective, 1, ws, st);
    if (method == CQ_BOUNDED) {
        cqk::SweepArgs a{};
        a.w = w; a.d = d; a.d_period = d_period;
        a.scales = scales; a.codes = codes; a.objective = objective; a.flags = flags;
        a.pscales = pooled_scales; a.pobjective = pooled_objective;
        a.fb_count = (int32_t*)ws;
        a.fb_list = (int32_t*)(ws + ALIGN);
        a.parts = (cqk::SlicePart*)(ws + ALIGN + round_up((size_t)n_groups * 4u));
        a.want_minimax = 1;
        a.want_pooled = (pooled_scales || pooled_objective) ? 1 : 0;
        return hip_status(cqk::launch_sweep(a, E, n_groups, st));
    }
    cqk::CandArgs c{};
    c.w = w; c.d = d; c.d_period = d_period; c.n_groups = n_groups;
    c.G = CQ_GROUP; c.qmin = -8; c.qmax = 7; c.start_ratio = 1.0f / 9.0f;
    c.scales = scales; c.codes = codes; c.objective = objective; c.flags = flags;
    c.tie_count = (int32_t*)ws;
    c.tie_list = (int32_t*)(ws + ALIGN);
    // groups whose direct candidates tied are decided by the exhaustive sweep, whose binary64
    // queue counter is cleared together with the tie counter
    uint8_t* sws = ws + ALIGN + round_up((size_t)n_groups * 4u);
    c.zero_also = (int32_t*)sws;
    hipError_t e = cqk::launch_candidate(c, E, st);
    if (e != hipSuccess) return CQ_EHIP;
    cqk::SweepArgs a{};
    a.w = w; a.d = d; a.d_period = d_period;
    a.list = c.tie_list; a.list_count = c.tie_count;
    a.scales = scales; a.codes = codes; a.objective = objective; a.flags = flags;
    a.fb_count = (int32_t*)sws;
    a.fb_list = (int32_t*)(sws + ALIGN);
    a.parts = (cqk::SlicePart*)(sws + ALIGN + round_up((size_t)n_groups * 4u));
    a.want_minimax = 1;
    a.want_pooled = 0;
    a.mark_fallback = 1;
    a.fb_zeroed = 1;
    return hip_status(cqk::launch_sweep(a, E, n_groups, st));
}

int32_t cq_quantize_groups_spec(const float* w, const float* d, int32_t group_len, int32_t qmin, int32_t qmax,
                                int64_t d_period, int32_t E, int64_t n_groups, int32_t method, uint16_t* scales,
                                int8_t* codes, double* objective, uint8_t* flags, uint16_t* pooled_scales,
                                double* pooled_objective, void* workspace, size_t workspace_bytes, void* stream) {
    if (!spec_ok(group_len, qmin, qmax)) return CQ_EINVAL;
    if (method != CQ_EXHAUSTIVE && method != CQ_CANDIDATE && method != CQ_BOUNDED) return CQ_EINVAL;
    if (group_len == CQ_GROUP && qmin == -8 && qmax == 7)
        return cq_quantize_groups(w, d, d_period, E, n_groups, method, scales, codes, objective, flags, pooled_scales,
                                  pooled_objective, workspace, workspace_bytes, stream);
    const bool cand = method == CQ_CANDIDATE && cand_spec_ok(group_len, qmin, qmax);
    if (method != CQ_EXHAUSTIVE && !cand) return CQ_EUNSUPPORTED;
    if (!groups_ok(w, d, d_period, E, n_groups, 4)) return CQ_EINVAL;
    if (n_groups > 0 && !scales) return CQ_EINVAL;
    if (n_groups > INT32_MAX) return CQ_EINVAL;
    if (cand && (pooled_scales || pooled_objective)) return CQ_EUNSUPPORTED;
    if (n_groups == 0) return CQ_OK;
    if (!workspace || workspace_bytes < cq_workspace_size(method, E, n_groups) || !aligned(workspace, ALIGN))
        return CQ_EWORKSPACE;
    hipStream_t st = (hipStream_t)stream;
    uint8_t* ws = (uint8_t*)workspace;
    if (!cand)
        return run_fullgrid(w, d, group_len, qmin, qmax, d_period, E, n_groups, scales, codes, objective, flags,
                            pooled_scales, pooled_objective, 1, ws, st);
    // the candidate solver; the groups whose direct candidates tied are decided by the full grid
    // (list mode), which takes every quantizer
    cqk::CandArgs c{};
    c.w = w; c.d = d; c.d_period = d_period; c.n_groups = n_groups;
    c.G = group_len; c.qmin = qmin; c.qmax = qmax;
    c.start_ratio = 1.0f / (float)((-qmin > qmax ? -qmin : qmax) + 1);
    c.scales = scales; c.codes = codes; c.objective = objective; c.flags = flags;
    c.tie_count = (int32_t*)ws;
    c.tie_list = (int32_t*)(ws + ALIGN);
    uint8_t* fws = ws + ALIGN + round_up((size_t)n_groups * 4u);  // sweep_ws(n_groups) bytes
    hipError_t e = cqk::launch_candidate(c, E, st);
    if (e != hipSuccess) return CQ_EHIP;
    cqk::FullArgs a{};
    a.w = w; a.d = d; a.d_period = d_period; a.G = group_len; a.qmin = qmin; a.qmax = qmax;
    a.ratio = cqk::fullgrid_ratio(group_len, qmin, qmax, E);
    a.scales = scales; a.codes = codes; a.objective = objective; a.flags = flags;
    a.want_minimax = 1;
    a.want_pooled = 0;
    a.fb_count = (int32_t*)fws;
    a.fb_list = (int32_t*)(fws + ALIGN);
    a.parts = (cqk::SlicePart*)(fws + full_ws(n_groups));
    a.list = c.tie_list;
    a.list_count = c.tie_count;
    a.flag_or = CQ_FLAG_FALLBACK;
    return hip_status(cqk::launch_fullgrid(a, E, n_groups, st));
}

int32_t cq_baseline_scales(const float* w, const float* d, int64_t d_period, int32_t E, int64_t n_groups,
                           int32_t which, uint16_t* scales, int8_t* codes, double* objective, void* workspace,
                           size_t workspace_bytes, void* stream) {
    hipStream_t st = (hipStream_t)stream;
    if (n_groups < 0 || n_groups > INT32_MAX) return CQ_EINVAL;
    if (which == CQ_ABSMAX) {
        if (n_groups == 0) return CQ_OK;
        if (!w || !scales || !aligned(w, 16) || (codes && !aligned(codes, 16))) return CQ_EINVAL;
        if (objective && !groups_ok(w, d, d_period, E, n_groups)) return CQ_EINVAL;
        return hip_status(cqk::launch_absmax(w, d, d_period, E, n_groups, scales, codes, objective, st));
    }
    if (which != CQ_POOLED_WMSE) return CQ_EINVAL;
    if (!groups_ok(w, d, d_period, E, n_groups)) return CQ_EINVAL;
    if (n_groups == 0) return CQ_OK;
    if (!scales) return CQ_EINVAL;
    const size_t need = cq_workspace_size(CQ_BOUNDED, E, n_groups);
    if (!workspace || workspace_bytes < need || !aligned(workspace, ALIGN)) return CQ_EWORKSPACE;
    uint8_t* ws = (uint8_t*)workspace;
    cqk::SweepArgs a{};
    a.w = w; a.d = d; a.d_period = d_period;
    a.codes = codes; a.pscales = scales; a.pobjective = objective;
    a.fb_count = (int32_t*)ws;
    a.fb_list = (int32_t*)(ws + ALIGN);
    a.parts = (cqk::SlicePart*)(ws + ALIGN + round_up((size_t)n_groups * 4u));
    a.want_minimax = 0;
    a.want_pooled = 1;
    return hip_status(cqk::launch_sweep(a, E, n_groups, st));
}

int32_t cq_baseline_scales_spec(const float* w, const float* d, int32_t group_len, int32_t qmin, int32_t qmax,
                                int64_t d_period, int32_t E, int64_t n_groups, int32_t which, uint16_t* scales,
                                int8_t* codes, double* objective, void* workspace, size_t workspace_bytes,
                                void* stream) {
    if (!spec_ok(group_len, qmin, qmax)) return CQ_EINVAL;
    if (group_len == CQ_GROUP && qmin == -8 && qmax == 7)
        return cq_baseline_scales(w, d, d_period, E, n_groups, which, scales, codes, objective, workspace,
                                  workspace_bytes, stream);
    hipStream_t st = (hipStream_t)stream;
    if (n_groups < 0 || n_groups > INT32_MAX) return CQ_EINVAL;
    if (which == CQ_ABSMAX) {
        if (qmax < 1) return CQ_EINVAL;  // the largest magnitude maps to the largest positive code
        if (n_groups == 0) return CQ_OK;
        if (!w || !scales || !aligned(w, 4)) return CQ_EINVAL;
        if (objective && !groups_ok(w, d, d_period, E, n_groups, 4)) return CQ_EINVAL;
        return hip_status(cqk::launch_absmax_spec(w, d, d_period, group_len, qmin, qmax, E, n_groups, scales, codes,
                                                  objective, st));
    }
    if (which != CQ_POOLED_WMSE) return CQ_EINVAL;
    if (!groups_ok(w, d, d_period, E, n_groups, 4)) return CQ_EINVAL;
    if (n_groups == 0) return CQ_OK;
    if (!scales) return CQ_EINVAL;
    if (!workspace || workspace_bytes < cq_workspace_size(CQ_EXHAUSTIVE, E, n_groups) || !aligned(workspace, ALIGN))
        return CQ_EWORKSPACE;
    // the full grid's pooled policy alone; its codes are those of the pooled scale
    return run_fullgrid(w, d, group_len, qmin, qmax, d_period, E, n_groups, nullptr, codes, nullptr, nullptr, scales,
                        objective, 0, (uint8_t*)workspace, st);
}

int32_t cq_pack_gptq_v1(const int8_t* codes, const uint16_t* grp_scales, int64_t out, int64_t in,
                        int32_t* qweight, uint16_t* scales, void* stream) {
    if (out < 0 || in < 0 || in % CQ_GROUP != 0) return CQ_EINVAL;
    if (out == 0 || in == 0) return CQ_OK;
    if (!codes || !grp_scales || !qweight || !scales) return CQ_EINVAL;
    if (!aligned(codes, 16) || !aligned(grp_scales, 2) || !aligned(qweight, 4) || !aligned(scales, 2))
        return CQ_EINVAL;
    if (in / CQ_GROUP > 65535 || (out + 63) / 64 > INT32_MAX) return CQ_EINVAL;
    return hip_status(cqk::launch_pack(codes, grp_scales, out, in, qweight, scales, (hipStream_t)stream));
}

int32_t cq_pack_gptq_v1_spec(const int8_t* codes, const uint16_t* grp_scales, int64_t out, int64_t in, int32_t bits,
                             int32_t group_len, int32_t* qweight, uint16_t* scales, void* stream) {
    if (bits != 2 && bits != 4 && bits != 8) return CQ_EINVAL;
    if (group_len < 1 || group_len > CQ_MAX_GROUP) return CQ_EINVAL;
    if (out < 0 || in < 0 || in % group_len != 0 || in % (32 / bits) != 0) return CQ_EINVAL;
    if (out == 0 || in == 0) return CQ_OK;
    if (!codes || !grp_scales || !qweight || !scales) return CQ_EINVAL;
    if (!aligned(codes, 4) || !aligned(grp_scales, 2) || !aligned(qweight, 4) || !aligned(scales, 2))
        return CQ_EINVAL;
    if ((in + 127) / 128 > 65535 || (out + 63) / 64 > INT32_MAX || (in / group_len) > INT64_MAX / (out + 1) ||
        ((in / group_len) * out + 255) / 256 > INT32_MAX)
        return CQ_EINVAL;
    return hip_status(cqk::launch_pack_spec(codes, grp_scales, out, in, bits, group_len, qweight, scales,
                                            (hipStream_t)stream));
}

int32_t cq_pack_gptq_v1_multi(const int8_t* codes, const uint16_t* grp_scales, int32_t n_mats, const int64_t* outs,
                              const int64_t* ins, int32_t* qweight, uint16_t* scales, void* stream) {
    if (n_mats < 0 || n_mats > CQ_MAX_PACK_MATRICES) return CQ_EINVAL;
    if (n_mats == 0) return CQ_OK;
    if (!outs || !ins) return CQ_EINVAL;
    cqk::PackShapes m{};
    m.n = n_mats;
    int64_t elems = 0, tiles = 0;
    for (int32_t k = 0; k < n_mats; ++k) {
        const int64_t o = outs[k], i = ins[k];
        if (o < 0 || i < 0 || i % CQ_GROUP != 0 || o > INT32_MAX || i > INT32_MAX) return CQ_EINVAL;
        if (i / CQ_GROUP > 65535) return CQ_EINVAL;
        m.out[k] = (int32_t)o;
        m.in[k] = (int32_t)i;
        elems += o * i;
        tiles += (o + 63) / 64 * (i / CQ_GROUP);
        if (elems > ((int64_t)1 << 46)) return CQ_EINVAL;
    }
    if (tiles == 0) return CQ_OK;
    if (!codes || !grp_scales || !qweight || !scales) return CQ_EINVAL;
    if (!aligned(codes, 16) || !aligned(grp_scales, 2) || !aligned(qweight, 4) || !aligned(scales, 2))
        return CQ_EINVAL;
    return hip_status(cqk::launch_pack_multi(codes, grp_scales, m, qweight, scales, (hipStream_t)stream));
}

size_t cq_proxy_workspace_size(int64_t n_groups) {
    return n_groups < 0 ? 0 : round_up((size_t)n_groups * 8u);
}

int32_t cq_proxy_worst_env_wmse_multi(const float* w, const float* d_eval, int64_t d_period, int32_t E,
                                      int64_t n_groups, int32_t n_policies, const uint16_t* scales,
                                      const int64_t* module_offsets, int32_t n_modules, double* module_mean,
                                      double* macro, double* per_group, void* workspace, size_t workspace_bytes,
                                      void* stream) {
    if (!groups_ok(w, d_eval, d_period, E, n_groups)) return CQ_EINVAL;
    if (n_policies < 1 || n_policies > CQ_MAX_POLICIES) return CQ_EINVAL;
    if (n_modules < 1 || !module_offsets || !module_mean || !macro) return CQ_EINVAL;
    if (n_groups > 0 && !scales) return CQ_EINVAL;
    if ((n_groups + 15) / 16 > INT32_MAX || n_groups > INT64_MAX / 8 / n_policies) return CQ_EINVAL;
    if (!per_group) {
        if (!workspace || workspace_bytes < cq_proxy_workspace_size(n_groups * n_policies) ||
            !aligned(workspace, ALIGN))
            return CQ_EWORKSPACE;
        per_group = (double*)workspace;
    } else if (!aligned(per_group, 8)) {
        return CQ_EINVAL;
    }
    return hip_status(cqk::launch_proxy(w, d_eval, d_period, E, n_groups, n_policies, scales, module_offsets,
                                        n_modules, module_mean, macro, per_group, (hipStream_t)stream));
}

int32_t cq_proxy_worst_env_wmse_multi_spec(const float* w, const float* d_eval, int32_t group_len, int32_t qmin,
                                           int32_t qmax, int64_t d_period, int32_t E, int64_t n_groups,
                                           int32_t n_policies, const uint16_t* scales, const int64_t* module_offsets,
                                           int32_t n_modules, double* module_mean, double* macro, double* per_group,
                                           void* workspace, size_t workspace_bytes, void* stream) {
    if (!spec_ok(group_len, qmin, qmax)) return CQ_EINVAL;
    if (group_len == CQ_GROUP && qmin == -8 && qmax == 7)
        return cq_proxy_worst_env_wmse_multi(w, d_eval, d_period, E, n_groups, n_policies, scales, module_offsets,
                                             n_modules, module_mean, macro, per_group, workspace, workspace_bytes,
                                             stream);
    if (!groups_ok(w, d_eval, d_period, E, n_groups, 4)) return CQ_EINVAL;
    if (n_policies < 1 || n_policies > CQ_MAX_POLICIES) return CQ_EINVAL;
    if (n_modules < 1 || !module_offsets || !module_mean || !macro) return CQ_EINVAL;
    if (n_groups > 0 && !scales) return CQ_EINVAL;
    if ((n_groups + 15) / 16 > INT32_MAX || n_groups > INT64_MAX / 8 / n_policies) return CQ_EINVAL;
    if (!per_group) {
        if (!workspace || workspace_bytes < cq_proxy_workspace_size(n_groups * n_policies) ||
            !aligned(workspace, ALIGN))
            return CQ_EWORKSPACE;
        per_group = (double*)workspace;
    } else if (!aligned(per_group, 8)) {
        return CQ_EINVAL;
    }
    return hip_status(cqk::launch_proxy_spec(w, d_eval, d_period, group_len, qmin, qmax, E, n_groups, n_policies,
                                             scales, module_offsets, n_modules, module_mean, macro, per_group,
                                             (hipStream_t)stream));
}

int32_t cq_proxy_worst_env_wmse(const float* w, const float* d_eval, int64_t d_period, int32_t E, int64_t n_groups,
                                const uint16_t* scales, const int64_t* module_offsets, int32_t n_modules,
                                double* module_mean, double* macro, double* per_group, void* workspace,
                                size_t workspace_bytes, void* stream) {
    return cq_proxy_worst_env_wmse_multi(w, d_eval, d_period, E, n_groups, 1, scales, module_offsets, n_modules,
                                         module_mean, macro, per_group, workspace, workspace_bytes, stream);
}

int32_t cq_w4a16_matmul(const uint16_t* x, const int32_t* qweight, const uint16_t* scales, int64_t M, int64_t out,
                        int64_t in, float* y, void* stream) {
    if (M < 0 || out < 0 || in < 0 || in % CQ_GROUP != 0) return CQ_EINVAL;
    if (M == 0 || out == 0) return CQ_OK;
    if (in == 0) return CQ_EINVAL;
    if ((M + 63) / 64 > 65535 || (out + 63) / 64 > INT32_MAX) return CQ_EINVAL;
    if (!x || !qweight || !scales || !y) return CQ_EINVAL;
    if (!aligned(x, 16) || !aligned(qweight, 4) || !aligned(scales, 2) || !aligned(y, 4)) return CQ_EINVAL;
    return hip_status(cqk::launch_w4a16(x, qweight, scales, M, out, in, y, (hipStream_t)stream));
}

int32_t cq_w4a16_linear(const void* x, int64_t ldx, int32_t x_type, const int32_t* qweight, const uint16_t* scales,
                        const void* bias, const void* residual, int64_t ldr, int32_t activation, int32_t gated,
                        int64_t M, int64_t out, int64_t in, void* y, int64_t ldy, int32_t y_type, void* stream) {
    if ((x_type != CQ_BF16 && x_type != CQ_F16) || (y_type != x_type && y_type != CQ_F32)) return CQ_EINVAL;
    if (activation < CQ_ACT_NONE || activation > CQ_ACT_GELU_TANH || (gated != 0 && gated != 1)) return CQ_EINVAL;
    if (M < 0 || out < 0 || in <= 0 || in % CQ_GROUP != 0) return CQ_EINVAL;
    if (M > INT32_MAX || out > (gated ? INT32_MAX / 2 : INT32_MAX) || in > (int64_t)1 << 24) return CQ_EINVAL;
    if (M == 0 || out == 0) return CQ_OK;
    if (!x || !qweight || !scales || !y) return CQ_EINVAL;
    if (ldx < in || ldx % 8 != 0 || ldy < out || (residual && ldr < out)) return CQ_EINVAL;
    if (!aligned(x, 16) || !aligned(qweight, 4) || !aligned(scales, 2) || !aligned(bias, 2) || !aligned(residual, 2) ||
        !aligned(y, y_type == CQ_F32 ? 4 : 2))
        return CQ_EINVAL;
    cqk::LinearArgs a{};
    a.x = (const uint16_t*)x; a.qw = qweight; a.scales = scales;
    a.bias = (const uint16_t*)bias; a.residual = (const uint16_t*)residual; a.y = y;
    a.M = M; a.out = out; a.in = in; a.ldx = ldx; a.ldr = ldr; a.ldy = ldy;
    a.x_f16 = x_type == CQ_F16; a.y_f32 = y_type == CQ_F32; a.act = activation; a.gated = gated;
    return hip_status(cqk::launch_linear(a, (hipStream_t)stream));
}

int32_t cq_kv_block_map(const int32_t* ctx_len, const int32_t* new_len, int32_t n_requests, int32_t page_size,
                        const int32_t* free_pages, const int32_t* n_free, int32_t free_capacity, int32_t* block_table,
                        int64_t table_stride, int32_t max_pages, int32_t max_tokens, int32_t* cu_q, int32_t* kv_len,
                        int32_t* slots, int32_t* positions, int32_t* status, int32_t* n_left, void* stream) {
    if (n_requests < 0 || n_requests > CQ_MAX_REQUESTS || page_size < 1 || max_pages < 1 || max_tokens < 0)
        return CQ_EINVAL;
    if ((int64_t)max_pages * page_size > INT32_MAX || table_stride < max_pages || free_capacity < 0) return CQ_EINVAL;
    if (!n_free || !n_left || n_left == n_free || !cu_q) return CQ_EINVAL;
    if (n_requests > 0 && (!ctx_len || !new_len || !block_table || !kv_len || !status)) return CQ_EINVAL;
    if (n_requests > 0 && (kv_len == ctx_len || kv_len == new_len || status == ctx_len || status == new_len))
        return CQ_EINVAL;
    if ((free_capacity > 0 && !free_pages) || (max_tokens > 0 && (!slots || !positions))) return CQ_EINVAL;
    const void* all[] = {ctx_len, new_len, free_pages, n_free, block_table, cu_q, kv_len, slots, positions, status,
                         n_left};
    for (const void* p : all)
        if (!aligned(p, 4)) return CQ_EINVAL;
    cqk::BlockMapArgs a{};
    a.ctx = ctx_len; a.add = new_len; a.free_pages = free_pages; a.n_free = n_free; a.table = block_table;
    a.cu = cu_q; a.kv_len = kv_len; a.slots = slots; a.positions = positions; a.status = status; a.n_left = n_left;
    a.table_stride = table_stride; a.R = n_requests; a.page = page_size; a.free_cap = free_capacity;
    a.max_pages = max_pages; a.max_tokens = max_tokens;
    return hip_status(cqk::launch_block_map(a, (hipStream_t)stream));
}

int32_t cq_kv_cache_write(const void* k, int64_t k_token_stride, int64_t k_head_stride, const void* v,
                          int64_t v_token_stride, int64_t v_head_stride, void* k_cache, void* v_cache,
                          int64_t page_stride, int64_t head_stride, int64_t row_stride, int32_t n_pages,
                          int32_t page_size, int32_t kv_heads, int32_t head_dim, const int32_t* slots,
                          int32_t n_tokens, void* stream) {
    if (n_tokens < 0 || n_pages < 0 || kv_heads < 1 || page_size < 1 || head_dim < 1) return CQ_EINVAL;
    if ((k_token_stride | k_head_stride | v_token_stride | v_head_stride | page_stride | head_stride | row_stride) < 0)
        return CQ_EINVAL;
    if (n_tokens == 0 || n_pages == 0) return CQ_OK;
    if (!k || !v || !k_cache || !v_cache || !slots) return CQ_EINVAL;
    if (!aligned(k, 2) || !aligned(v, 2) || !aligned(k_cache, 2) || !aligned(v_cache, 2) || !aligned(slots, 4))
        return CQ_EINVAL;
    cqk::CacheWriteArgs a{};
    a.k = (const uint16_t*)k; a.v = (const uint16_t*)v; a.kc = (uint16_t*)k_cache; a.vc = (uint16_t*)v_cache;
    a.slots = slots; a.k_tok = k_token_stride; a.k_head = k_head_stride; a.v_tok = v_token_stride;
    a.v_head = v_head_stride; a.c_page = page_stride; a.c_head = head_stride; a.c_row = row_stride;
    a.n_slots = (int64_t)n_pages * page_size; a.T = n_tokens; a.H = kv_heads; a.D = head_dim; a.page = page_size;
    return hip_status(cqk::launch_cache_write(a, (hipStream_t)stream));
}

static bool attention_sizes_ok(int32_t T, int32_t R, int32_t max_q, int32_t max_kv, int32_t H, int32_t Hkv, int32_t D) {
    return T >= 0 && R >= 0 && max_q >= 0 && max_kv >= 0 && Hkv >= 1 && H >= Hkv && H % Hkv == 0 && H <= 65535 &&
           D >= 8 && D <= CQ_MAX_HEAD_DIM && D % 8 == 0 && (int64_t)T * H <= INT32_MAX && R <= 65535;
}

size_t cq_paged_attention_workspace_size(int32_t n_tokens, int32_t n_requests, int32_t max_q, int32_t max_kv,
                                         int32_t heads, int32_t kv_heads, int32_t head_dim) {
    if (!attention_sizes_ok(n_tokens, n_requests, max_q, max_kv, heads, kv_heads, head_dim)) return 0;
    return (size_t)cqk::attention_ws(n_requests, n_tokens, max_q, max_kv, heads, kv_heads, head_dim) * 4u;
}

int32_t cq_paged_attention(const cq_paged_attention_args* args, void* workspace, size_t workspace_bytes,
                           void* stream) {
    if (!args) return CQ_EINVAL;
    const cq_paged_attention_args& p = *args;
    if (p.type != CQ_BF16 && p.type != CQ_F16) return CQ_EINVAL;
    if (!attention_sizes_ok(p.n_tokens, p.n_requests, p.max_q, p.max_kv, p.heads, p.kv_heads, p.head_dim))
        return CQ_EINVAL;
    if (p.page_size < 1 || p.n_pages < 0 || p.max_pages < 0 || p.table_stride < p.max_pages) return CQ_EINVAL;
    if ((int64_t)p.max_pages * p.page_size > (int64_t)1 << 30) return CQ_EINVAL;
    if ((p.causal != 0 && p.causal != 1) || p.window < 0 || (p.window > 0 && !p.causal)) return CQ_EINVAL;
    if (!(p.scale - p.scale == 0.0f)) return CQ_EINVAL;
    if ((p.q_token_stride | p.q_head_stride | p.out_token_stride | p.out_head_stride | p.page_stride | p.head_stride |
         p.row_stride) < 0 ||
        (p.q_token_stride | p.q_head_stride | p.out_token_stride | p.out_head_stride | p.page_stride | p.head_stride |
         p.row_stride) % 8 != 0)
        return CQ_EINVAL;
    if (p.n_tokens == 0) return CQ_OK;
    if (!p.q || !p.out || !p.cu_q) return CQ_EINVAL;
    if (p.n_requests > 0 && !p.kv_len) return CQ_EINVAL;
    if (p.n_pages > 0 && p.max_pages > 0 && p.n_requests > 0 && (!p.k_cache || !p.v_cache || !p.block_table))
        return CQ_EINVAL;
    if (!aligned(p.q, 16) || !aligned(p.k_cache, 16) || !aligned(p.v_cache, 16) || !aligned(p.out, 16) ||
        !aligned(p.block_table, 4) || !aligned(p.cu_q, 4) || !aligned(p.kv_len, 4) || !aligned(p.lse, 4))
        return CQ_EINVAL;
    if (!cqk::attention_fits(p.n_requests, p.n_tokens, p.max_q, p.max_kv, p.heads, p.kv_heads, p.head_dim))
        return CQ_EUNSUPPORTED;
    const size_t need = cq_paged_attention_workspace_size(p.n_tokens, p.n_requests, p.max_q, p.max_kv, p.heads,
                                                          p.kv_heads, p.head_dim);
    if (need && (!workspace || workspace_bytes < need || !aligned(workspace, ALIGN))) return CQ_EWORKSPACE;
    cqk::AttentionArgs a{};
    a.q = (const uint16_t*)p.q; a.kc = (const uint16_t*)p.k_cache; a.vc = (const uint16_t*)p.v_cache;
    a.out = (uint16_t*)p.out; a.lse = p.lse; a.table = p.block_table; a.cu = p.cu_q; a.kv_len = p.kv_len;
    a.q_tok = p.q_token_stride; a.q_head = p.q_head_stride; a.o_tok = p.out_token_stride; a.o_head = p.out_head_stride;
    a.c_page = p.page_stride; a.c_head = p.head_stride; a.c_row = p.row_stride; a.table_stride = p.table_stride;
    a.page = p.page_size; a.n_pages = p.n_pages; a.max_pages = p.max_pages;
    a.R = p.n_requests; a.T = p.n_tokens; a.max_q = p.max_q; a.max_kv = p.max_kv;
    a.H = p.heads; a.Hkv = p.kv_heads; a.D = p.head_dim; a.causal = p.causal; a.window = p.window;
    a.f16 = p.type == CQ_F16; a.scale = p.scale; a.ws = (float*)workspace;
    return hip_status(cqk::launch_attention(a, (hipStream_t)stream));
}

size_t cq_diagonals_workspace_size(int32_t E, int64_t T, int64_t in) {
    if (E < 1 || E > CQ_MAX_ENVS || T < 1 || in < CQ_GROUP || in % CQ_GROUP != 0 || in > (int64_t)1 << 24) return 0;
    return round_up((size_t)E * (size_t)cqk::diag_chunks(E, T, in) * (size_t)in * 8u) + round_up((size_t)E * (size_t)in * 8u);
}

int32_t cq_environment_diagonals(const uint16_t* x, int32_t E, int64_t T, int64_t in, float* d, void* workspace,
                                 size_t workspace_bytes, void* stream) {
    if (E < 1 || E > CQ_MAX_ENVS || T < 1 || in < CQ_GROUP || in % CQ_GROUP != 0 || in > (int64_t)1 << 24)
        return CQ_EINVAL;
    if (!x || !d || !aligned(x, 16) || !aligned(d, 4)) return CQ_EINVAL;
    const size_t need = cq_diagonals_workspace_size(E, T, in);
    if (!workspace || workspace_bytes < need || !aligned(workspace, ALIGN)) return CQ_EWORKSPACE;
    uint8_t* ws = (uint8_t*)workspace;
    double* part = (double*)ws;
    double* msq = (double*)(ws + round_up((size_t)E * (size_t)cqk::diag_chunks(E, T, in) * (size_t)in * 8u));
    return hip_status(cqk::launch_diagonals(x, E, T, in, d, part, msq, (hipStream_t)stream));
}

size_t cq_heldout_workspace_size(int32_t n_boot, int32_t n_modules) {
    if (n_boot < 0 || n_modules < 1) return 0;
    return round_up((size_t)(n_boot + 1) * (size_t)n_modules * 8u) + round_up((size_t)n_boot * 8u) +
           round_up((size_t)n_boot * 4u);
}

int32_t cq_heldout_compare(const double* pa, const double* pb, int64_t n_groups, const int64_t* module_offsets,
                           int32_t n_modules, const int32_t* boot_idx, int32_t n_boot, double alpha,
                           int64_t* counts, double* effect, double* boot, double* ci, void* workspace,
                           size_t workspace_bytes, void* stream) {
    if (n_groups < 0 || n_modules < 1 || n_boot < 0 || n_boot > CQ_MAX_BOOT) return CQ_EINVAL;
    if (!(alpha > 0.0 && alpha < 1.0)) return CQ_EINVAL;
    if (n_groups > 0 && (!pa || !pb || !aligned(pa, 8) || !aligned(pb, 8))) return CQ_EINVAL;
    if (!module_offsets || !aligned(module_offsets, 8) || !counts || !effect || !ci) return CQ_EINVAL;
    if (n_boot > 0 && (!boot_idx || !boot || !aligned(boot_idx, 4))) return CQ_EINVAL;
    if ((int64_t)(n_boot + 1) * n_modules > INT32_MAX) return CQ_EINVAL;
    if (!workspace || workspace_bytes < cq_heldout_workspace_size(n_boot, n_modules) || !aligned(workspace, ALIGN))
        return CQ_EWORKSPACE;
    uint8_t* ws = (uint8_t*)workspace;
    double* mm = (double*)ws;
    double* reps = (double*)(ws + round_up((size_t)(n_boot + 1) * (size_t)n_modules * 8u));
    int32_t* rank = (int32_t*)((uint8_t*)reps + round_up((size_t)n_boot * 8u));
    return hip_status(cqk::launch_heldout(pa, pb, n_groups, module_offsets, n_modules, boot_idx, n_boot, alpha,
                                          counts, effect, boot, ci, mm, reps, rank, (hipStream_t)stream));
}

int32_t cq_probe_valu_fma(int32_t iters, int32_t blocks, int32_t mode, float* out, uint64_t* clocks,
                          double* wall_clock_hz, void* stream) {
    if (iters < 1 || blocks < 1 || (mode < 0 || mode > 2) || !out || !clocks || !wall_clock_hz) return CQ_EINVAL;
    int dev = 0, khz = 0;
    if (hipGetDevice(&dev) != hipSuccess) return CQ_EHIP;
    if (hipDeviceGetAttribute(&khz, hipDeviceAttributeWallClockRate, dev) != hipSuccess || khz <= 0) return CQ_EHIP;
    *wall_clock_hz = 1e3 * (double)khz;
    return hip_status(cqk::launch_fma_probe(iters, blocks, mode, out, clocks, (hipStream_t)stream));
}

}  // extern "C"
